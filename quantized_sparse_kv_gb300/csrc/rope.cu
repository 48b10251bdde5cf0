// Rotary positions (kv_rope) of q, k and, copied, v of one projection.
//
// Mathematics. Pair i of a token at position pos turns by 2 pi phi, phi the
// fraction of pos * f_i / (2 pi). f_i / (2 pi) comes as a 64-bit binary
// fraction of a turn, so the product modulo 2^64 (ordinary wrapping integer
// arithmetic, negative positions included) is phi with the table's error times
// |pos|: its entries are made from doubles, below 2^-53 turns a position, so the
// farthest position (2^31) is off by less than 2^-22 turns and one of 2^20 by 2^-33;
// no 64-bit floating point is used on the device. phi goes to fp32 as a signed fraction
// (relative error 2^-24) and through sincospif; the two products of a pair are
// fp32, rounded once to the output type.
//
// What bounds it: memory. Every element is read and written once, 16 bytes a
// thread and head. The sine and cosine of a thread's pairs are made once and
// serve every head it visits; the heads of a token are spread over `splits`
// threads only as far as the call needs threads to cover the card (a decoding
// step takes one head a thread, a prompt several). The first heads' loads are
// issued before a thread makes its sines.
// Measured: q, k and v rows of a projection, 2 x 8,192 tokens x 20 heads of 128 bf16
// (151 MB moved): 29.0 us, 5.2 TB/s, what a plain copy of this size reaches; 3 x
// 1,023 x 18 fp32 heads (57 MB): 12.9 us, a copy 16 us; 64 tokens: 4.6 us, the launch.
#include <math.h>

#include <algorithm>

#include "kvq_internal.h"

namespace kvq {
namespace {

constexpr int kRopeThreads = 256;
// Heads a thread has in flight (16 bytes each in bf16, 32 in fp32), and the CTAs
// per SM that its registers are held to. The prompt above: 1 head 33.9 us, 2 heads
// 29.0, 3 heads in two CTAs 36.9; two heads in three or five CTAs 33-35. fp32, 57 MB:
// 1 head 12.9, 2 heads 14.3.
template <typename T>
constexpr int kRopeHeads = sizeof(T) == 2 ? 2 : 1;
constexpr int kRopeCtas = 4;

struct RopeArgs {
  RopeTensors t;
  int n, D, rot;      // tokens, head dim, rotary dim
  int tokens;         // batch * n
  int units, splits;  // 8-feature units per head; threads that share a token's heads
  const uint64_t *turns;
  const int32_t *pos;
  float amp, sign;
  KernelCtl ctl;
};

// Eight elements of a row, as loaded and as floats.
template <typename T>
struct Raw8;
template <>
struct Raw8<float> {
  float4 a, b;
};
template <>
struct Raw8<__nv_bfloat16> {
  uint4 w;
};
__device__ __forceinline__ void load8(const float *p, Raw8<float> &r) {
  r.a = *reinterpret_cast<const float4 *>(p);
  r.b = *reinterpret_cast<const float4 *>(p + 4);
}
__device__ __forceinline__ void load8(const __nv_bfloat16 *p, Raw8<__nv_bfloat16> &r) {
  r.w = *reinterpret_cast<const uint4 *>(p);
}
__device__ __forceinline__ void to_floats(const Raw8<float> &r, float (&x)[8]) {
  x[0] = r.a.x, x[1] = r.a.y, x[2] = r.a.z, x[3] = r.a.w;
  x[4] = r.b.x, x[5] = r.b.y, x[6] = r.b.z, x[7] = r.b.w;
}
__device__ __forceinline__ void to_floats(const Raw8<__nv_bfloat16> &r, float (&x)[8]) {
  const uint32_t u[4] = {r.w.x, r.w.y, r.w.z, r.w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(u[i] << 16);
    x[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void store8(float *p, const float (&x)[8]) {
  *reinterpret_cast<float4 *>(p) = make_float4(x[0], x[1], x[2], x[3]);
  *reinterpret_cast<float4 *>(p + 4) = make_float4(x[4], x[5], x[6], x[7]);
}
__device__ __forceinline__ void store8(__nv_bfloat16 *p, const float (&x)[8]) {
  *reinterpret_cast<uint4 *>(p) = make_uint4(pack_bf2(x[0], x[1]), pack_bf2(x[2], x[3]),
                                             pack_bf2(x[4], x[5]), pack_bf2(x[6], x[7]));
}

// cos and sin (times the amplitude; sin negated for the inverse) of a phase
// given in 2^-64 turns.
__device__ __forceinline__ void phase_cs(const RopeArgs &a, int pair, int pos, float &c, float &s) {
  const uint64_t phase = static_cast<uint64_t>(static_cast<int64_t>(pos)) * a.turns[pair];
  // signed fraction of a turn, in half turns: [-1, 1]
  const float x = static_cast<float>(static_cast<int64_t>(phase)) * 0x1p-63f;
  float sn, cs;
  sincospif(x, &sn, &cs);
  c = cs * a.amp;
  s = sn * a.amp * a.sign;
}

// Input and output of head h (counted over all tensors) of token (b, t).
template <typename T>
__device__ __forceinline__ void head_ptrs(const RopeArgs &a, int h, int b, int t, const T *&in,
                                          T *&out, bool &rotate) {
  int k = 0;
  while (k + 1 < a.t.n && h >= a.t.heads[k]) h -= a.t.heads[k++];
  in = static_cast<const T *>(a.t.in[k]) + b * a.t.sb[k] + h * a.t.sh[k] + t * a.t.st[k];
  out = static_cast<T *>(a.t.out[k]) +
        ((static_cast<int64_t>(b) * a.t.heads[k] + h) * a.n + t) * a.D;
  rotate = a.t.rotate[k] != 0;
}

// kHalf: a unit below rot / 16 is 8 pairs (features 8u.. and rot/2 + 8u..),
// the units after them 8 features that pass through (rot is a multiple of
// 16). Otherwise (interleaved pairs) a unit is 8 consecutive features.
template <typename T, bool kHalf>
__global__ void __launch_bounds__(kRopeThreads, kRopeCtas) rope_kernel(const RopeArgs a) {
  wait_prior_grid();
  allow_next_grid();
  const int64_t id = static_cast<int64_t>(blockIdx.x) * kRopeThreads + threadIdx.x;
  const int per = a.units * a.splits;
  const int64_t token = id / per;
  if (token >= a.tokens) return;
  const int rem = static_cast<int>(id - token * per);
  const int u = rem % a.units, h0 = rem / a.units;
  const int b = static_cast<int>(token / a.n), t = static_cast<int>(token - static_cast<int64_t>(b) * a.n);
  const int pos = in_bounds(a.ctl, a.pos + token, 4) ? a.pos[token] : 0;
  constexpr int kPairs = kHalf ? 8 : 4;
  const int half = a.rot / 2;
  const int d0 = kHalf ? (u < a.rot / 16 ? 8 * u : a.rot + 8 * (u - a.rot / 16)) : 8 * u;
  const bool pairs = kHalf ? u < a.rot / 16 : d0 < a.rot;
  // Heads go kRopeHeads at a time, all loads of a batch in flight together; the
  // first batch's are issued before the sines and cosines are made.
  Raw8<T> rx[kRopeHeads<T>], ry[kHalf ? kRopeHeads<T> : 1];
  T *out[kRopeHeads<T>];
  bool turn[kRopeHeads<T>];
  auto load = [&](int h) {
#pragma unroll
    for (int k = 0; k < kRopeHeads<T>; ++k, h += a.splits) {
      out[k] = nullptr;
      if (h >= a.t.total_heads) continue;
      const T *in;
      head_ptrs(a, h, b, t, in, out[k], turn[k]);
      if (!in_bounds(a.ctl, in, a.D * sizeof(T)) || !in_bounds(a.ctl, out[k], a.D * sizeof(T))) {
        out[k] = nullptr;
        continue;
      }
      load8(in + d0, rx[k]);
      if (kHalf && pairs) load8(in + d0 + half, ry[kHalf ? k : 0]);
    }
  };
  load(h0);
  float c[kPairs], s[kPairs];
#pragma unroll
  for (int i = 0; i < kPairs; ++i) {
    c[i] = 1.0f;
    s[i] = 0.0f;
    const int p = kHalf ? d0 + i : d0 / 2 + i;
    if (pairs && p < half && in_bounds(a.ctl, a.turns + p, 8)) phase_cs(a, p, pos, c[i], s[i]);
  }
#pragma unroll 1
  for (int h = h0;;) {
#pragma unroll
    for (int k = 0; k < kRopeHeads<T>; ++k) {
      if (!out[k]) continue;
      float x[8], y[8];
      to_floats(rx[k], x);
      if (kHalf && pairs) {
        to_floats(ry[kHalf ? k : 0], y);
        if (turn[k]) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float x0 = x[i], x1 = y[i];
            x[i] = x0 * c[i % kPairs] - x1 * s[i % kPairs];
            y[i] = x0 * s[i % kPairs] + x1 * c[i % kPairs];
          }
        }
        store8(out[k] + d0 + half, y);
      } else if (!kHalf && pairs && turn[k]) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float x0 = x[2 * i], x1 = x[2 * i + 1];
          if (d0 / 2 + i < half) {
            x[2 * i] = x0 * c[i] - x1 * s[i];
            x[2 * i + 1] = x0 * s[i] + x1 * c[i];
          }
        }
      }
      store8(out[k] + d0, x);
    }
    h += kRopeHeads<T> * a.splits;
    if (h >= a.t.total_heads) break;
    load(h);
  }
}

// Half layout with a rotary dim that is no multiple of 16: one thread per pair
// or passed feature (units of one element), the same arithmetic (134 MB: 52.6 us
// at rotary dim 120, 26.0 us in the kernel above at 128).
template <typename T>
__global__ void __launch_bounds__(kRopeThreads) rope_pair_kernel(const RopeArgs a) {
  wait_prior_grid();
  allow_next_grid();
  const int64_t id = static_cast<int64_t>(blockIdx.x) * kRopeThreads + threadIdx.x;
  const int per = a.units * a.splits;
  const int64_t token = id / per;
  if (token >= a.tokens) return;
  const int rem = static_cast<int>(id - token * per);
  const int u = rem % a.units, h0 = rem / a.units;
  const int b = static_cast<int>(token / a.n), t = static_cast<int>(token - static_cast<int64_t>(b) * a.n);
  const int half = a.rot / 2;
  const bool pair = u < half;
  float c = 1.0f, s = 0.0f;
  if (pair && in_bounds(a.ctl, a.pos + token, 4) && in_bounds(a.ctl, a.turns + u, 8))
    phase_cs(a, u, a.pos[token], c, s);
  for (int h = h0; h < a.t.total_heads; h += a.splits) {
    const T *in;
    T *out;
    bool rotate;
    head_ptrs(a, h, b, t, in, out, rotate);
    if (!in_bounds(a.ctl, in, a.D * sizeof(T)) || !in_bounds(a.ctl, out, a.D * sizeof(T))) continue;
    if (!pair) {
      out[half + u] = in[half + u];  // unit half + k is feature rot + k
      continue;
    }
    const T r0 = in[u], r1 = in[u + half];
    if (rotate) {
      const float x0 = load_f32(&r0), x1 = load_f32(&r1);
      store_from_f32(out + u, x0 * c - x1 * s);
      store_from_f32(out + u + half, x0 * s + x1 * c);
    } else {
      out[u] = r0;
      out[u + half] = r1;
    }
  }
}

template <typename T>
int launch_typed(RopeArgs &a, bool half_layout, int num_sms, cudaStream_t s) {
  const bool scalar = half_layout && a.rot % 16 != 0;
  a.units = scalar ? a.D - a.rot / 2
                   : half_layout ? a.rot / 16 + (a.D - a.rot) / 8 : a.D / 8;
  // Threads per token: enough for about 2,048 a SM over the whole call, at
  // most one head each.
  const int64_t want = static_cast<int64_t>(num_sms) * 2048;
  const int64_t base = static_cast<int64_t>(a.tokens) * a.units;
  a.splits = static_cast<int>(
      std::max<int64_t>(1, std::min<int64_t>(a.t.total_heads, (want + base - 1) / base)));
  const int64_t threads = base * a.splits;
  const dim3 grid(static_cast<unsigned>((threads + kRopeThreads - 1) / kRopeThreads));
  if (scalar)
    launch_dependent(rope_pair_kernel<T>, grid, dim3(kRopeThreads), 0, s, a);
  else if (half_layout)
    launch_dependent(rope_kernel<T, true>, grid, dim3(kRopeThreads), 0, s, a);
  else
    launch_dependent(rope_kernel<T, false>, grid, dim3(kRopeThreads), 0, s, a);
  return 1;
}

}  // namespace

int launch_rope(const RopeTensors &t, int dtype, int batch, int n, int D, int rot, int layout,
                const uint64_t *turns, float amplitude, int inverse, const int32_t *positions,
                const KernelCtl &ctl, int num_sms, cudaStream_t s) {
  RopeArgs a;
  a.t = t;
  a.n = n;
  a.D = D;
  a.rot = rot;
  a.tokens = batch * n;
  a.turns = turns;
  a.pos = positions;
  a.amp = amplitude;
  a.sign = inverse ? -1.0f : 1.0f;
  a.ctl = ctl;
  const bool half_layout = layout == KVQ_ROPE_HALF;
  return dtype == KVQ_F32 ? launch_typed<float>(a, half_layout, num_sms, s)
                          : launch_typed<__nv_bfloat16>(a, half_layout, num_sms, s);
}

// f_i / (2 pi) of every pair as a 64-bit binary fraction of a turn. Host code.
bool rope_turns(int rot, double base, const kvq_rope_scaling *sc, uint64_t *turns, float *amp) {
  constexpr double kTwoPi = 6.283185307179586476925286766559;
  const int kind = sc ? sc->kind : KVQ_ROPE_NONE;
  if (!(base > 1.0) || !std::isfinite(base)) return false;
  if (kind < KVQ_ROPE_NONE || kind > KVQ_ROPE_BANDS) return false;
  if (kind != KVQ_ROPE_NONE && (!(sc->factor >= 1.0) || !std::isfinite(sc->factor))) return false;
  if (kind == KVQ_ROPE_BASE && rot < 4) return false;
  if (kind >= KVQ_ROPE_RAMP) {
    if (!(sc->original > 0.0) || !std::isfinite(sc->original) || !std::isfinite(sc->p0) ||
        !std::isfinite(sc->p1))
      return false;
    if (kind == KVQ_ROPE_RAMP && !(sc->p1 > 0.0 && sc->p0 > sc->p1)) return false;
    if (kind == KVQ_ROPE_BANDS && !(sc->p0 >= 0.0 && sc->p1 > sc->p0)) return false;
  }
  const double r = rot;
  double b = base;
  if (kind == KVQ_ROPE_BASE) b = base * std::pow(sc->factor, r / (r - 2.0));
  if (!std::isfinite(b)) return false;
  double lo = 0.0, hi = 1.0;
  *amp = 1.0f;
  if (kind == KVQ_ROPE_RAMP) {
    auto pair_of = [&](double t) {
      return r * std::log(sc->original / (kTwoPi * t)) / (2.0 * std::log(b));
    };
    // (both ends inside the range: a context so long, or so short, that every
    // pair lies on one side of the ramp must not turn it around)
    lo = std::min(r - 1.0, std::max(0.0, std::floor(pair_of(sc->p0))));
    hi = std::min(r - 1.0, std::max(0.0, std::ceil(pair_of(sc->p1))));
    if (hi == lo) hi += 0.001;  // a step instead of a ramp
    *amp = static_cast<float>(0.1 * std::log(sc->factor) + 1.0);
  }
  for (int i = 0; i < rot / 2; ++i) {
    double f = std::pow(b, -2.0 * i / r);
    if (kind == KVQ_ROPE_LINEAR) {
      f /= sc->factor;
    } else if (kind == KVQ_ROPE_RAMP) {
      const double w = std::min(1.0, std::max(0.0, (i - lo) / (hi - lo)));
      f = f / sc->factor * w + f * (1.0 - w);
    } else if (kind == KVQ_ROPE_BANDS) {
      const double w = std::min(
          1.0, std::max(0.0, (sc->original * f / kTwoPi - sc->p0) / (sc->p1 - sc->p0)));
      f = f / sc->factor * (1.0 - w) + f * w;
    }
    turns[i] = static_cast<uint64_t>(std::ldexp(f / kTwoPi, 64));  // f <= 1: below 2^62
  }
  return true;
}

}  // namespace kvq
