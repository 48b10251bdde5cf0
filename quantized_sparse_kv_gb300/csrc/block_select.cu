// Block summaries of a packed cache (kv_block_summary) and the choice of
// blocks from them (kv_select_blocks).
//
// Mathematics. A block's summary is the mean of its dequantized keys, rounded
// to int8 with one scale: with c the codes of a 32-token group and s its
// per-channel scale the group's sum is fl(s * sum c), sum c an integer; the
// groups' sums are added in order. A query row is rounded to int8 the same
// way, the product of the two code vectors is an integer below 2^24, and the
// score is two fp32 multiplications. Nothing depends on the order of the
// additions, so the chosen blocks are a function of the inputs alone.
//
// What bounds them. The summary reads 20 D bytes of K codes and scales per
// group and writes D + 4 per block: memory. Scoring reads D + 4 bytes per
// block (of 64 tokens at D = 128: 1/78 of its K and V) for 2 heads * D integer operations;
// choosing is a radix selection over one score row and bound by latency. Measured,
// D = 128, blocks of 64: summaries of 32 x 2 x 131,072 tokens (671 MB of codes and
// scales) 108 us, 6.4 TB/s; their values (17 MB read, 67 written) 14 us; scores of
// 8 heads over 64 x 2,046 blocks (17.3 MB, cold) 8.1 us and the choice of 32 of them
// 5.0 us. Scores and choice in one kernel for this many blocks (a cluster per query
// token, scores kept in shared memory) took 6 us longer than the two.
#include <math_constants.h>

#include <algorithm>

#include "int4_dequant.cuh"
#include "kvq_internal.h"

namespace kvq {
namespace {

// fl(x / s) rounded to an integer in [-127, 127], 0 for a zero scale. |x / s| passes
// 127.5 only where s = fl(max / 127) is subnormal, rounded by up to a third of itself.
__device__ __forceinline__ int int8_code(float x, float s) {
  return s > 0.0f ? max(-127, min(127, __float2int_rn(__fdiv_rn(x, s)))) : 0;
}

struct SummaryArgs {
  const uint8_t *k_codes;
  const float *k_scales;
  int8_t *codes;
  float *scales;
  int D, cut, Gk, Gs;      // Gs: K groups per unit (stride)
  int m;                   // groups per block
  int first, blocks, cap;  // blocks [first, blocks) are computed; cap: stride
  long units;
  KernelCtl ctl;
};

// ------------------------------------------------------------------ D = 128
// One warp per block. A lane reads 16 bytes (32 channels) of a token row, so
// four loads of a warp take a whole group's codes (2 KB) and one more its
// scales. Nibbles are summed as bytes: two masks split a word into its even
// and odd channels, four tokens a lane and three lane exchanges give the 32
// tokens' sums (a byte holds 16 tokens' worth, 240; the last exchange is on
// 16-bit halves). Each exchange also halves what a lane keeps, so a lane ends
// with the four channels whose scales it loaded.
constexpr int kSumWarps = 8;

// Sums of the codes of one group in this lane's channels: 32 (lane & 3) +
// 16 b2 + 8 b3 + 4 b4 + 0..3, b2..b4 the lane's upper bits.
__device__ __forceinline__ int4 group_sums(const uint4 (&w)[4], int lane) {
  uint32_t lo[4] = {0, 0, 0, 0}, hi[4] = {0, 0, 0, 0};  // word j: channels 8j + 0,2,4,6 / 1,3,5,7
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t x[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      lo[j] += x[j] & 0x0F0F0F0Fu;
      hi[j] += (x[j] >> 4) & 0x0F0F0F0Fu;
    }
  }
  const bool b2 = lane & 4, b3 = lane & 8, b4 = lane & 16;
  uint32_t l2[2], h2[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) {  // keep words 0,1 (b2 = 0) or 2,3
    l2[j] = (b2 ? lo[2 + j] : lo[j]) + __shfl_xor_sync(0xffffffffu, b2 ? lo[j] : lo[2 + j], 4);
    h2[j] = (b2 ? hi[2 + j] : hi[j]) + __shfl_xor_sync(0xffffffffu, b2 ? hi[j] : hi[2 + j], 4);
  }
  const uint32_t l1 = (b3 ? l2[1] : l2[0]) + __shfl_xor_sync(0xffffffffu, b3 ? l2[0] : l2[1], 8);
  const uint32_t h1 = (b3 ? h2[1] : h2[0]) + __shfl_xor_sync(0xffffffffu, b3 ? h2[0] : h2[1], 8);
  // widen: channels (0, 2) and (4, 6) of the word, (1, 3) and (5, 7)
  const uint32_t la = prmt(l1, 0u, 0x4140u), lb = prmt(l1, 0u, 0x4342u);
  const uint32_t ha = prmt(h1, 0u, 0x4140u), hb = prmt(h1, 0u, 0x4342u);
  const uint32_t e = (b4 ? lb : la) + __shfl_xor_sync(0xffffffffu, b4 ? la : lb, 16);
  const uint32_t o = (b4 ? hb : ha) + __shfl_xor_sync(0xffffffffu, b4 ? ha : hb, 16);
  // 32 tokens of code + 8: padding tokens hold code 0
  return make_int4(static_cast<int>(e & 0xffffu) - 256, static_cast<int>(o & 0xffffu) - 256,
                   static_cast<int>(e >> 16) - 256, static_cast<int>(o >> 16) - 256);
}

template <int M>
__global__ void __launch_bounds__(kSumWarps * 32) summary128_kernel(const SummaryArgs a) {
  wait_prior_grid();
  allow_next_grid();
  const int lane = threadIdx.x & 31;
  const long per = a.blocks - a.first;
  const long id = static_cast<long>(blockIdx.x) * kSumWarps + (threadIdx.x >> 5);
  if (id >= per * a.units) return;
  const long u = id / per;
  const int blk = a.first + static_cast<int>(id - u * per);
  const int g0 = blk * M;
  const int ch = 32 * (lane & 3) + ((lane & 4) << 2) + (lane & 8) + ((lane & 16) >> 2);
  uint4 w[M][4];
  float4 sc[M];
#pragma unroll
  for (int g = 0; g < M; ++g) {
    const bool have = g0 + g < a.Gk;
    const long gi = u * a.Gs + g0 + g;
    const uint8_t *p = a.k_codes + gi * 2048 + 16 * lane;
    const float *s = a.k_scales + gi * 128 + ch;
#pragma unroll
    for (int i = 0; i < 4; ++i)  // lane reads token 8i + lane / 4, bytes 16 (lane & 3)..
      w[g][i] = have && in_bounds(a.ctl, p + 512 * i, 16)
                    ? __ldcs(reinterpret_cast<const uint4 *>(p + 512 * i))
                    : make_uint4(0x88888888u, 0x88888888u, 0x88888888u, 0x88888888u);
    sc[g] = have && in_bounds(a.ctl, s, 16) ? __ldcs(reinterpret_cast<const float4 *>(s))
                                            : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  }
  float acc[4];
#pragma unroll
  for (int g = 0; g < M; ++g) {
    const int4 c = group_sums(w[g], lane);
    const float p[4] = {__fmul_rn(sc[g].x, static_cast<float>(c.x)),
                        __fmul_rn(sc[g].y, static_cast<float>(c.y)),
                        __fmul_rn(sc[g].z, static_cast<float>(c.z)),
                        __fmul_rn(sc[g].w, static_cast<float>(c.w))};
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[j] = g == 0 ? p[j] : __fadd_rn(acc[j], p[j]);
  }
  const float tokens = static_cast<float>(min(32 * M, a.cut - 32 * M * blk));
  float mx = 0.0f;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    acc[j] = __fdiv_rn(acc[j], tokens);
    mx = fmaxf(mx, fabsf(acc[j]));
  }
  const float scale = __fdiv_rn(warp_max(mx), 127.0f);
  uint32_t out = 0u;
#pragma unroll
  for (int j = 0; j < 4; ++j)
    out |= (static_cast<uint32_t>(int8_code(acc[j], scale)) & 0xffu) << (8 * j);
  const long row = u * a.cap + blk;
  if (in_bounds(a.ctl, a.codes + row * 128 + ch, 4))
    *reinterpret_cast<uint32_t *>(a.codes + row * 128 + ch) = out;
  if (lane == 0 && in_bounds(a.ctl, a.scales + row, 4)) a.scales[row] = scale;
}

// ------------------------------------------------------------------ any D
// One warp per block again, a lane per 4 bytes (8 channels) of a token row and as
// many rows at once as fit the warp (a power of two). A word's channels are summed
// as bytes for 16 tokens (240 at most) and as 16-bit halves from there on, the row
// lanes' sums meet in the first row's, which hold eight channels each then.
// (D = 64, 84 MB: 34.2 us; the kernel above takes 16.8 us for as much at D = 128.)
template <int kRows>  // token rows at once
__global__ void __launch_bounds__(kSumWarps * 32) summary_kernel(const SummaryArgs a) {
  wait_prior_grid();
  allow_next_grid();
  const int lane = threadIdx.x & 31, D = a.D;
  const long per = a.blocks - a.first;
  const long id = static_cast<long>(blockIdx.x) * kSumWarps + (threadIdx.x >> 5);
  if (id >= per * a.units) return;
  const long u = id / per;
  const int blk = a.first + static_cast<int>(id - u * per);
  const int pieces = D / 8;  // lanes per token row
  const int row = lane / pieces, piece = lane - row * pieces;
  const bool on = row < kRows;
  float acc[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) acc[i] = 0.0f;
  for (int g = 0; g < a.m && blk * a.m + g < a.Gk; ++g) {
    const long gi = u * a.Gs + blk * a.m + g;
    const uint8_t *p = a.k_codes + (gi * 32 + row) * (D / 2) + 4 * piece;
    const float *s = a.k_scales + gi * D + 8 * piece;
    // the channels' scales are on their way while the codes are summed
    float4 s0 = make_float4(0.0f, 0.0f, 0.0f, 0.0f), s1 = s0;
    if (row == 0 && in_bounds(a.ctl, s, 32)) {
      s0 = *reinterpret_cast<const float4 *>(s);
      s1 = *reinterpret_cast<const float4 *>(s + 4);
    }
    uint32_t sum[4] = {0u, 0u, 0u, 0u};  // sum[k]: channels k (low half) and k + 4
    constexpr int kTokens = kRows == 1 ? 16 : 32 / kRows;  // of a lane, in bytes
#pragma unroll
    for (int t0 = 0; t0 < 32; t0 += kTokens * kRows) {
      uint32_t lo = 0u, hi = 0u, x[kTokens];  // bytes: channels 0, 2, 4, 6 and 1, 3, 5, 7
#pragma unroll
      for (int t = 0; t < kTokens; ++t) {
        const uint8_t *w = p + (t0 + t * kRows) * (D / 2);
        x[t] = on && in_bounds(a.ctl, w, 4) ? __ldcs(reinterpret_cast<const uint32_t *>(w))
                                            : 0x88888888u;
      }
#pragma unroll
      for (int t = 0; t < kTokens; ++t) {
        lo += x[t] & 0x0F0F0F0Fu;
        hi += (x[t] >> 4) & 0x0F0F0F0Fu;
      }
      sum[0] += lo & 0x00FF00FFu;
      sum[1] += hi & 0x00FF00FFu;
      sum[2] += (lo >> 8) & 0x00FF00FFu;
      sum[3] += (hi >> 8) & 0x00FF00FFu;
    }
#pragma unroll
    for (int r = kRows / 2; r > 0; r /= 2) {
#pragma unroll
      for (int k = 0; k < 4; ++k) sum[k] += __shfl_down_sync(0xffffffffu, sum[k], r * pieces);
    }
    const float sc[8] = {s0.x, s0.y, s0.z, s0.w, s1.x, s1.y, s1.z, s1.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      // 32 tokens of code + 8: padding tokens hold code 0
      const int c = static_cast<int>((sum[i & 3] >> (i < 4 ? 0 : 16)) & 0xffffu) - 256;
      const float part = __fmul_rn(sc[i], static_cast<float>(c));
      acc[i] = g == 0 ? part : __fadd_rn(acc[i], part);
    }
  }
  const float tokens = static_cast<float>(min(32 * a.m, a.cut - 32 * a.m * blk));
  float mx = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    acc[i] = __fdiv_rn(acc[i], tokens);
    mx = row == 0 ? fmaxf(mx, fabsf(acc[i])) : 0.0f;
  }
  const float scale = __fdiv_rn(warp_max(mx), 127.0f);
  const long at = u * a.cap + blk;
  if (lane == 0 && in_bounds(a.ctl, a.scales + at, 4)) a.scales[at] = scale;
  int8_t *o = a.codes + at * D + 8 * piece;
  if (row != 0 || !in_bounds(a.ctl, o, 8)) return;
  uint32_t out[2] = {0u, 0u};
#pragma unroll
  for (int i = 0; i < 8; ++i)
    out[i >> 2] |= (static_cast<uint32_t>(int8_code(acc[i], scale)) & 0xffu) << (8 * (i & 3));
  *reinterpret_cast<uint2 *>(o) = make_uint2(out[0], out[1]);
}

// ------------------------------------------------------------------ values
// code * scale of every summary from `first` on, dense: a thread takes four codes of
// four rows at a time, so a warp stores 512 consecutive bytes and keeps eight
// loads in flight. Memory: 1.25 D bytes read, 4 D written per block.
constexpr int kValThreads = 256, kValRows = 4;

__global__ void __launch_bounds__(kValThreads) values_kernel(const SummaryArgs a, float *out) {
  wait_prior_grid();
  allow_next_grid();
  const int D4 = a.D / 4, rows = a.blocks - a.first;
  const int per = kValThreads / D4;  // rows the CTA takes at once
  const int piece = threadIdx.x % D4, r0 = threadIdx.x / D4;
  if (r0 >= per) return;
  for (long u = blockIdx.y; u < a.units; u += gridDim.y) {
    const int base = static_cast<int>(blockIdx.x) * per * kValRows + r0;
    uint32_t c[kValRows];
    float s[kValRows];
#pragma unroll
    for (int i = 0; i < kValRows; ++i) {
      const int row = base + i * per;
      const long from = u * a.cap + a.first + row;
      const bool ok = row < rows && in_bounds(a.ctl, a.codes + from * a.D + 4 * piece, 4) &&
                      in_bounds(a.ctl, a.scales + from, 4);
      c[i] = ok ? *reinterpret_cast<const uint32_t *>(a.codes + from * a.D + 4 * piece) : 0u;
      s[i] = ok ? a.scales[from] : 0.0f;
    }
#pragma unroll
    for (int i = 0; i < kValRows; ++i) {
      const int row = base + i * per;
      float4 *o = reinterpret_cast<float4 *>(out + (u * rows + row) * a.D) + piece;
      if (row >= rows || !in_bounds(a.ctl, o, 16)) continue;
      __stcs(o, make_float4(
                    static_cast<float>(static_cast<int8_t>(c[i] & 0xffu)) * s[i],
                    static_cast<float>(static_cast<int8_t>(c[i] >> 8 & 0xffu)) * s[i],
                    static_cast<float>(static_cast<int8_t>(c[i] >> 16 & 0xffu)) * s[i],
                    static_cast<float>(static_cast<int8_t>(c[i] >> 24)) * s[i]));
    }
  }
}

// ------------------------------------------------------------------ scores
struct SelectArgs {
  const int8_t *codes;
  const float *scales;
  const void *q;
  int q_dtype;
  int D, Hkv, G, n_q;   // G: query heads per KV head
  int blocks, cap, top_k, sink;
  float *scores;        // [unit][n_q][stride], stride = blocks rounded up to 4
  int stride;
  int32_t *selected;
  KernelCtl ctl;
};

constexpr int kScoreThreads = 128;
constexpr int kMaxGroup = 64;  // query heads per KV head

// The rows of q of a (unit, query token) as int8 to shared memory, G heads padded with
// zeros to a multiple of eight: a warp per row, its largest magnitude first.
template <int kPer, int kThreads>  // features a lane holds, threads of the CTA
__device__ __forceinline__ void round_queries(const SelectArgs &a, long u, int iq, int D,
                                              int8_t *qs, float *sq) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int h = warp; h < (a.G + 7) / 8 * 8; h += kThreads / 32) {
    const long row = (u * a.G + h) * a.n_q + iq;  // [batch][q_heads][n_q], q head = kv * G + h
    float x[kPer], mx = 0.0f;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int d = lane + 32 * i;
      x[i] = 0.0f;
      if (h < a.G && d < D) {
        if (a.q_dtype == KVQ_F32) {
          const float *p = static_cast<const float *>(a.q) + row * D + d;
          if (in_bounds(a.ctl, p, 4)) x[i] = *p;
        } else {
          const uint16_t *p = static_cast<const uint16_t *>(a.q) + row * D + d;
          if (in_bounds(a.ctl, p, 2)) x[i] = bf16_to_f32(*p);
        }
      }
      mx = fmaxf(mx, fabsf(x[i]));
    }
    const float s = __fdiv_rn(warp_max(mx), 127.0f);
    if (lane == 0) sq[h] = h < a.G ? s : 0.0f;
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (lane + 32 * i < D) qs[h * D + lane + 32 * i] = static_cast<int8_t>(int8_code(x[i], s));
  }
}

// D = 128, on the int8 tensor cores: a warp's MMA takes 16 blocks x 8 heads x 32
// features, so four of them and four 16-byte loads a lane score 16 blocks. Lane
// (g, t) holds bytes 16t .. 16t + 15 and 64 + 16t .. of rows g and g + 8 and of head g:
// the MMA's feature order is permuted the same way on both sides, which a dot
// product does not see. A warp's two tiles of 16 blocks are in flight while q is
// rounded. (Byte dot products: a thread per block 34.0 us for select and attend over
// 32 sequences of 131,072 tokens, eight lanes a block 30.1, this 28.4.)
constexpr int kScoreTiles = 2;

__device__ __forceinline__ void mma_s8(int (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                       uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+r"(c[0]), "+r"(c[1]), "+r"(c[2]), "+r"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Rows g and g + 8 of a warp's tiles, blocks first + 8 r.
struct ScoreRows {
  uint4 k[2 * kScoreTiles][2];
  float s[2 * kScoreTiles];
};
__device__ __forceinline__ void load_rows(const SelectArgs &a, long u, int first, int t,
                                          ScoreRows &x) {
#pragma unroll
  for (int r = 0; r < 2 * kScoreTiles; ++r) {
    const long row = u * a.cap + first + 8 * r;
    const bool have = first + 8 * r < a.blocks && in_bounds(a.ctl, a.codes + row * 128, 128) &&
                      in_bounds(a.ctl, a.scales + row, 4);
    const uint4 *p = reinterpret_cast<const uint4 *>(a.codes + row * 128) + t;
    x.k[r][0] = have ? p[0] : make_uint4(0u, 0u, 0u, 0u);
    x.k[r][1] = have ? p[4] : make_uint4(0u, 0u, 0u, 0u);
    x.s[r] = have ? a.scales[row] : 0.0f;
  }
}
// Their scores (in every lane of a row).
__device__ __forceinline__ void score_rows(const SelectArgs &a, const ScoreRows &x,
                                           const int8_t *qs, const float *sq, int first, int g,
                                           int t, float (&best)[2 * kScoreTiles]) {
#pragma unroll
  for (int r = 0; r < 2 * kScoreTiles; ++r) best[r] = -CUDART_INF_F;
#pragma unroll 1
  for (int h0 = 0; h0 < a.G; h0 += 8) {
    const uint4 *qp = reinterpret_cast<const uint4 *>(qs + (h0 + g) * 128) + t;
    const uint4 q0 = qp[0], q1 = qp[4];
    const float s0 = sq[h0 + 2 * t], s1 = sq[h0 + 2 * t + 1];
    const bool on0 = h0 + 2 * t < a.G, on1 = h0 + 2 * t + 1 < a.G;
#pragma unroll
    for (int i = 0; i < kScoreTiles; ++i) {
      const uint4(&lo)[2] = x.k[2 * i], (&hi)[2] = x.k[2 * i + 1];
      int c[4] = {0, 0, 0, 0};
      mma_s8(c, lo[0].x, hi[0].x, lo[0].y, hi[0].y, q0.x, q0.y);
      mma_s8(c, lo[0].z, hi[0].z, lo[0].w, hi[0].w, q0.z, q0.w);
      mma_s8(c, lo[1].x, hi[1].x, lo[1].y, hi[1].y, q1.x, q1.y);
      mma_s8(c, lo[1].z, hi[1].z, lo[1].w, hi[1].w, q1.z, q1.w);
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const float sb = x.s[2 * i + r];
        const float x0 = __fmul_rn(__fmul_rn(s0, sb), static_cast<float>(c[2 * r]));
        const float x1 = __fmul_rn(__fmul_rn(s1, sb), static_cast<float>(c[2 * r + 1]));
        if (on0) best[2 * i + r] = fmaxf(best[2 * i + r], x0);
        if (on1) best[2 * i + r] = fmaxf(best[2 * i + r], x1);
      }
    }
  }
#pragma unroll
  for (int r = 0; r < 2 * kScoreTiles; ++r) {
    best[r] = fmaxf(best[r], __shfl_xor_sync(0xffffffffu, best[r], 1));
    best[r] = fmaxf(best[r], __shfl_xor_sync(0xffffffffu, best[r], 2));
    if (first + 8 * r < a.sink) best[r] = CUDART_INF_F;
  }
}

__global__ void __launch_bounds__(kScoreThreads) block_scores128_kernel(const SelectArgs a) {
  wait_prior_grid();
  allow_next_grid();
  __shared__ __align__(16) int8_t qs[kMaxGroup * 128];
  __shared__ float sq[kMaxGroup];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
  const int uq = blockIdx.y;  // unit * n_q + query token
  const long u = uq / a.n_q;
  const int first = blockIdx.x * kScoreThreads + 16 * kScoreTiles * warp + g;
  ScoreRows x;
  load_rows(a, u, first, t, x);
  round_queries<4, kScoreThreads>(a, u, uq - static_cast<int>(u) * a.n_q, 128, qs, sq);
  __syncthreads();
  float best[2 * kScoreTiles];
  score_rows(a, x, qs, sq, first, g, t, best);
#pragma unroll
  for (int r = 0; r < 2 * kScoreTiles; ++r) {
    const int blk = first + 8 * r;
    float *o = a.scores + static_cast<long>(uq) * a.stride + blk;
    if (t == 0 && blk < a.blocks && in_bounds(a.ctl, o, 4)) *o = best[r];
  }
}

// Any D: one thread per block, its row read 16 bytes at a time, q read by broadcast.
__global__ void __launch_bounds__(kScoreThreads) block_scores_kernel(const SelectArgs a) {
  wait_prior_grid();
  allow_next_grid();
  extern __shared__ __align__(16) int8_t qs[];  // [ceil(G / 8) * 8][D]
  __shared__ float sq[kMaxGroup];
  const int D = a.D;
  const int uq = blockIdx.y;  // unit * n_q + query token
  const long u = uq / a.n_q;
  const int iq = uq - static_cast<int>(u) * a.n_q;
  round_queries<8, kScoreThreads>(a, u, iq, D, qs, sq);
  __syncthreads();
  const int blk = blockIdx.x * kScoreThreads + threadIdx.x;
  if (blk >= a.blocks) return;
  const long brow = u * a.cap + blk;
  float score = -CUDART_INF_F;
  if (in_bounds(a.ctl, a.codes + brow * D, D) && in_bounds(a.ctl, a.scales + brow, 4)) {
    const float sb = a.scales[brow];
    const uint4 *kp = reinterpret_cast<const uint4 *>(a.codes + brow * D);
    for (int h0 = 0; h0 < a.G; h0 += 8) {
      int dot[8] = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll 4
      for (int c = 0; c < D / 16; ++c) {
        const uint4 k = kp[c];
#pragma unroll
        for (int h = 0; h < 8; ++h) {
          const int4 q = *reinterpret_cast<const int4 *>(qs + (h0 + h) * D + 16 * c);
          dot[h] = __dp4a(static_cast<int>(k.x), q.x, dot[h]);
          dot[h] = __dp4a(static_cast<int>(k.y), q.y, dot[h]);
          dot[h] = __dp4a(static_cast<int>(k.z), q.z, dot[h]);
          dot[h] = __dp4a(static_cast<int>(k.w), q.w, dot[h]);
        }
      }
#pragma unroll
      for (int h = 0; h < 8; ++h)
        if (h0 + h < a.G)
          score = fmaxf(score, __fmul_rn(__fmul_rn(sq[h0 + h], sb), static_cast<float>(dot[h])));
    }
  }
  float *o = a.scores + static_cast<long>(uq) * a.stride + blk;
  if (in_bounds(a.ctl, o, 4)) *o = blk < a.sink ? CUDART_INF_F : score;
}

// ------------------------------------------------------------------ selection
// One CTA per (unit, query token): radix selection of the top_k-th largest
// score over order-preserving keys (8 bits a round, histogram in shared
// memory), then the blocks above it and the lowest-numbered ones equal to it
// are written in increasing order. The rounds end as soon as a whole digit is
// taken, which with scores that differ is after two or three. Up to kSelThreads *
// kSelKeys blocks every thread keeps the keys of consecutive blocks in
// registers, so one prefix sum places the output; more blocks go through the
// same code in pieces of that many, re-read from the workspace.
constexpr int kSelThreads = 256;
constexpr int kSelKeys = 8;

// Larger score, larger key; -0 counts as +0.
__device__ __forceinline__ uint32_t order_key(float x) {
  const uint32_t b = __float_as_uint(x + 0.0f);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}

// Exclusive prefix sum of v over the CTA and its total. Two copies of warp_sums,
// used in turn (`turn`), spare the barrier before the next scan.
__device__ __forceinline__ int cta_scan(int v, int (*warp_sums)[kSelThreads / 32], int turn,
                                        int &total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) warp_sums[turn & 1][warp] = x;
  __syncthreads();
  int before = 0;
  total = 0;
#pragma unroll
  for (int w = 0; w < kSelThreads / 32; ++w) {
    const int s = warp_sums[turn & 1][w];
    if (w < warp) before += s;
    total += s;
  }
  return before + x - v;
}

// Keys of blocks base + kSelKeys * thread .. + 7 (0, below every key, past the last).
__device__ __forceinline__ void load_keys(const float *sc, int base, int blocks,
                                          uint32_t (&key)[kSelKeys]) {
  const int i = base + kSelKeys * static_cast<int>(threadIdx.x);
#pragma unroll
  for (int j = 0; j < kSelKeys; j += 4) {
    // (rows are padded to four scores; a padding score is not looked at)
    const float4 f = i + j < blocks ? *reinterpret_cast<const float4 *>(sc + i + j)
                                    : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    key[j] = i + j < blocks ? order_key(f.x) : 0u;
    key[j + 1] = i + j + 1 < blocks ? order_key(f.y) : 0u;
    key[j + 2] = i + j + 2 < blocks ? order_key(f.z) : 0u;
    key[j + 3] = i + j + 3 < blocks ? order_key(f.w) : 0u;
  }
}

// The k = top_k blocks of the score row sc (k < blocks) to out, by the whole CTA.
__device__ __forceinline__ void select_row(const SelectArgs &a, const float *sc, int32_t *out) {
  __shared__ int hist[2][256], warp_sums[2][kSelThreads / 32];
  __shared__ uint32_t s_prefix;
  __shared__ int s_left, s_whole;
  const int tid = threadIdx.x, k = a.top_k;
  constexpr int kPiece = kSelThreads * kSelKeys;
  const bool one = a.blocks <= kPiece;
  uint32_t key[kSelKeys];
  load_keys(sc, 0, a.blocks, key);
  uint32_t prefix = 0u, mask = 0u;
  int left = k;  // how many of the keys matching the prefix are to be taken
  int turn = 0;
  hist[0][tid] = 0;
  for (int shift = 24; shift >= 0; shift -= 8, ++turn) {
    int *h = hist[turn & 1];
    hist[(turn + 1) & 1][tid] = 0;
    __syncthreads();
    for (int base = 0; base < a.blocks; base += kPiece) {
      if (!one) load_keys(sc, base, a.blocks, key);
#pragma unroll
      for (int j = 0; j < kSelKeys; ++j)
        if (key[j] != 0u && (key[j] & mask) == prefix) atomicAdd(&h[(key[j] >> shift) & 255u], 1);
    }
    __syncthreads();
    // the digit at which the count from the top reaches `left`: thread i
    // counts the digits above 255 - i
    int total;
    const int c = h[255 - tid];
    const int above = cta_scan(c, warp_sums, turn, total);
    if (above < left && above + c >= left) {
      s_prefix = prefix | (static_cast<uint32_t>(255 - tid) << shift);
      s_left = left - above;
      s_whole = above + c == left;
    }
    __syncthreads();
    prefix = s_prefix;
    left = s_left;
    mask |= 255u << shift;
    if (s_whole) break;  // every key with this prefix is taken
  }
  // keys above the prefix all, keys with it the first `left`
  int written = 0, equal_before = 0;
  for (int base = 0; base < a.blocks; base += kPiece) {
    if (!one) load_keys(sc, base, a.blocks, key);
    int gt = 0, eq = 0;
#pragma unroll
    for (int j = 0; j < kSelKeys; ++j) {
      gt += (key[j] & mask) > prefix;
      eq += key[j] != 0u && (key[j] & mask) == prefix;
    }
    int total;
    ++turn;
    // one scan for both counts: at most kPiece of each, below 2^16
    const int both = cta_scan(gt | eq << 16, warp_sums, turn, total);
    int eq_rank = equal_before + (both >> 16);
    int pos = written + (both & 0xffff) + min(eq_rank, left) - min(equal_before, left);
#pragma unroll
    for (int j = 0; j < kSelKeys; ++j) {
      const bool above = (key[j] & mask) > prefix;
      const bool equal = key[j] != 0u && (key[j] & mask) == prefix;
      if ((above || (equal && eq_rank < left)) && pos < k) out[pos++] = base + kSelKeys * tid + j;
      if (equal) ++eq_rank;
    }
    const int eq_total = total >> 16;
    written += (total & 0xffff) + min(equal_before + eq_total, left) - min(equal_before, left);
    equal_before += eq_total;
  }
}

__global__ void __launch_bounds__(kSelThreads) select_kernel(const SelectArgs a) {
  wait_prior_grid();
  allow_next_grid();
  const long uq = blockIdx.x;
  const float *sc = a.scores + uq * a.stride;
  int32_t *out = a.selected + uq * a.top_k;
  if (!in_bounds(a.ctl, out, sizeof(int32_t) * a.top_k)) return;
  if (a.blocks <= a.top_k) {  // all of them, then -1
    for (int i = threadIdx.x; i < a.top_k; i += kSelThreads) out[i] = i < a.blocks ? i : -1;
    return;
  }
  if (!in_bounds(a.ctl, sc, sizeof(float) * a.stride)) return;
  select_row(a, sc, out);
}

// Few blocks, D = 128: scores and choice in one CTA per (unit, query token), the
// scores in shared memory. Against the two kernels (select and attend together, 8
// heads): 253 blocks of 160 query tokens 24.0 us (25.6), 508 of 64 19.3 (20.4), 510 of 2
// 13.0 (13.0); 1,016 blocks of 64 21.2 (21.8), of 128 27.2 (28.3), but 1,022 of 2 15.1
// (13.6) and 2,046 of 64 27.9 (25.9): one CTA's pass over the blocks has to be short, or
// the card full.
constexpr int kFewBlocks = 1024;
__host__ bool few_blocks(long units, int blocks) {
  return blocks <= (units < 64 ? kFewBlocks / 2 : kFewBlocks);
}

__global__ void __launch_bounds__(kSelThreads) score_select128_kernel(const SelectArgs a) {
  wait_prior_grid();
  allow_next_grid();
  __shared__ __align__(16) int8_t qs[kMaxGroup * 128];
  __shared__ __align__(16) float sc[kFewBlocks];
  __shared__ float sq[kMaxGroup];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
  const int uq = blockIdx.x;  // unit * n_q + query token
  const long u = uq / a.n_q;
  int32_t *out = a.selected + static_cast<long>(uq) * a.top_k;
  if (!in_bounds(a.ctl, out, sizeof(int32_t) * a.top_k)) return;
  ScoreRows x;
  int first = 16 * kScoreTiles * warp + g;
  load_rows(a, u, first, t, x);
  round_queries<4, kSelThreads>(a, u, uq - static_cast<int>(u) * a.n_q, 128, qs, sq);
  __syncthreads();
#pragma unroll 1
  for (;;) {
    float best[2 * kScoreTiles];
    score_rows(a, x, qs, sq, first, g, t, best);
#pragma unroll
    for (int r = 0; r < 2 * kScoreTiles; ++r)
      if (t == 0 && first + 8 * r < a.blocks) sc[first + 8 * r] = best[r];
    first += kSelThreads / 2 * kScoreTiles;  // 16 blocks a warp and tile
    if (first - g >= a.blocks) break;
    load_rows(a, u, first, t, x);
  }
  __syncthreads();
  select_row(a, sc, out);
}

}  // namespace

int launch_block_summary(const kvq_cache &c, const kvq_summary &sm, int first, int blocks,
                         const KernelCtl &ctl, cudaStream_t s) {
  const CacheDims d = dims_of(c);
  SummaryArgs a;
  a.k_codes = c.k_codes;
  a.k_scales = c.k_scales;
  a.codes = sm.codes;
  a.scales = sm.scales;
  a.D = d.D;
  a.cut = d.cut;
  a.Gk = d.Gk;
  a.Gs = d.Gs;
  a.m = sm.block / kGroup;
  a.first = first;
  a.blocks = blocks;
  a.cap = sm.cap_blocks;
  a.units = static_cast<long>(d.B) * d.Hkv;
  a.ctl = ctl;
  const long warps = a.units * (blocks - first);
  const dim3 grid(static_cast<unsigned>((warps + kSumWarps - 1) / kSumWarps)), block(kSumWarps * 32);
  if (d.D > 128)
    launch_dependent(summary_kernel<1>, grid, block, 0, s, a);
  else if (d.D == 96)
    launch_dependent(summary_kernel<2>, grid, block, 0, s, a);
  else if (d.D == 64)
    launch_dependent(summary_kernel<4>, grid, block, 0, s, a);
  else if (d.D == 32)
    launch_dependent(summary_kernel<8>, grid, block, 0, s, a);
  else if (a.m == 1)
    launch_dependent(summary128_kernel<1>, grid, block, 0, s, a);
  else if (a.m == 2)
    launch_dependent(summary128_kernel<2>, grid, block, 0, s, a);
  else
    launch_dependent(summary128_kernel<4>, grid, block, 0, s, a);
  return 1;
}

int launch_block_values(const kvq_cache &c, const kvq_summary &sm, int first, int blocks,
                        float *values, const KernelCtl &ctl, cudaStream_t s) {
  SummaryArgs a = {};
  a.codes = sm.codes;
  a.scales = sm.scales;
  a.D = c.head_dim;
  a.first = first;
  a.blocks = blocks;
  a.cap = sm.cap_blocks;
  a.units = static_cast<long>(c.batch) * c.kv_heads;
  a.ctl = ctl;
  const int rows = kValThreads / (a.D / 4) * kValRows;
  const dim3 grid(static_cast<unsigned>((blocks - first + rows - 1) / rows),
                  static_cast<unsigned>(std::min<long>(a.units, 65535)));
  launch_dependent(values_kernel, grid, dim3(kValThreads), 0, s, a, values);
  return 1;
}

size_t select_workspace_bytes(const kvq_cache &c, int blocks, int n_q) {
  return sizeof(float) * static_cast<size_t>(c.batch) * c.kv_heads * n_q * ((blocks + 3) / 4 * 4);
}

int launch_select_blocks(const kvq_cache &c, const kvq_summary &sm, int blocks, const void *q,
                         int q_dtype, int Hq, int n_q, int top_k, int n_sink, int32_t *selected,
                         void *ws, const KernelCtl &ctl, cudaStream_t s) {
  SelectArgs a;
  a.codes = sm.codes;
  a.scales = sm.scales;
  a.q = q;
  a.q_dtype = q_dtype;
  a.D = c.head_dim;
  a.Hkv = c.kv_heads;
  a.G = Hq / c.kv_heads;
  a.n_q = n_q;
  a.blocks = blocks;
  a.cap = sm.cap_blocks;
  a.top_k = top_k;
  a.sink = n_sink;
  a.scores = static_cast<float *>(ws);
  a.stride = (blocks + 3) / 4 * 4;
  a.selected = selected;
  a.ctl = ctl;
  const unsigned units = static_cast<unsigned>(c.batch) * c.kv_heads * n_q;
  int launches = 0;
  if (blocks > top_k && a.D == 128 && few_blocks(units, blocks)) {
    launch_dependent(score_select128_kernel, dim3(units), dim3(kSelThreads), 0, s, a);
    return 1;
  }
  if (blocks > top_k) {
    const size_t smem = static_cast<size_t>((a.G + 7) / 8 * 8) * a.D;
    const dim3 grid((blocks + kScoreThreads - 1) / kScoreThreads, units);
    if (a.D == 128)
      launch_dependent(block_scores128_kernel, grid, dim3(kScoreThreads), 0, s, a);
    else
      launch_dependent(block_scores_kernel, grid, dim3(kScoreThreads), smem, s, a);
    ++launches;
  }
  launch_dependent(select_kernel, dim3(units), dim3(kSelThreads), 0, s, a);
  return launches + 1;
}

int select_max_group() { return kMaxGroup; }

}  // namespace kvq
