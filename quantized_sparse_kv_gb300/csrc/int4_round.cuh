// Exact int4 codes without a division per element (the bf16 kv_pack path).
//
// The grouped int4 rule of the residual-window page ("KV殘差窗口", section
// 固定預算) as this library states it: scale = fl(amax / 7), code =
// clamp(rint(fl(x / scale)), -7, 7), the divisions correctly rounded in fp32
// and rint to nearest, ties to even. Here the quotient comes from the
// correctly rounded reciprocal r = fl(1 / s) and one correction step
// (Markstein, "Computation of elementary functions on the IBM RISC
// System/6000 processor", IBM J. Res. Dev. 34(1), 1990): q0 = fl(x r), the
// residual e = x - q0 s exact through an fma, q = fl(q0 + e r). Adding
// 1.5 * 2^23 + 8 then rounds q to an integer, ties to even, and leaves
// code + 8 in bits 0-3 (bits 4-7 zero). The scale is formed the same way from
// fl(1 / 7). The clamp never binds: |x| <= amax puts fl(x / s) below 7.5.
//
// Every function is host and device code with the same arithmetic on both
// (the device intrinsics are the IEEE operations the host performs), so the
// CPU tests compile this file and check it, on every bf16 pair (amax, x)
// with |x| <= amax, against the correctly rounded division: equal wherever
// recip_ok(amax) holds, which is what the kernels test before taking it.
#pragma once

#include <stdint.h>
#include <string.h>

#include <cmath>

namespace kvq {

__host__ __device__ __forceinline__ float mul_rn(float a, float b) {
#ifdef __CUDA_ARCH__
  return __fmul_rn(a, b);
#else
  return a * b;
#endif
}
__host__ __device__ __forceinline__ float add_rn(float a, float b) {
#ifdef __CUDA_ARCH__
  return __fadd_rn(a, b);
#else
  return a + b;
#endif
}
__host__ __device__ __forceinline__ float fma_rn(float a, float b, float c) {
#ifdef __CUDA_ARCH__
  return __fmaf_rn(a, b, c);
#else
  return std::fma(a, b, c);
#endif
}
__host__ __device__ __forceinline__ float rcp_rn(float s) {  // fl(1 / s)
#ifdef __CUDA_ARCH__
  return __frcp_rn(s);
#else
  return 1.0f / s;
#endif
}
__host__ __device__ __forceinline__ uint32_t bits_of(float f) {
#ifdef __CUDA_ARCH__
  return __float_as_uint(f);
#else
  uint32_t u;
  memcpy(&u, &f, 4);
  return u;
#endif
}

// A group maximum the reciprocal path handles: zero, or finite and at least
// 2^-100 (below about 2^-119.6 the residual of a near-tie is no longer exact).
__host__ __device__ __forceinline__ bool recip_ok(float amax) {
  return amax == 0.0f || (amax >= 0x1p-100f && amax <= 3.40282347e38f);
}

// fl(amax / 7) for amax with recip_ok(amax).
__host__ __device__ __forceinline__ float scale_recip(float amax) {
  constexpr float r7 = 1.0f / 7.0f;
  const float q0 = mul_rn(amax, r7);
  return fma_rn(fma_rn(-q0, 7.0f, amax), r7, q0);
}

// The reciprocal the codes use (0 for a zero scale, whose codes are all 0).
__host__ __device__ __forceinline__ float recip_of(float s) {
  return s == 0.0f ? 0.0f : rcp_rn(s);
}

// code + 8 in bits 0-3 of the result (bits 4-7 zero), for |x| <= amax.
__host__ __device__ __forceinline__ uint32_t code8_recip(float x, float s, float r) {
  const float q0 = mul_rn(x, r);
  const float q = fma_rn(fma_rn(-q0, s, x), r, q0);
  return bits_of(add_rn(q, 12582920.0f));  // 1.5 * 2^23 + 8
}

// For any fp32 value: code + 8 in bits 0-3 of c (bits 4-7 zero), for |x| <= amax with
// recip_ok(amax), s = fl(amax / 7) and r = fl(1 / s) -- unless the answer is false. The
// product fl(x r) is off the true quotient by at most 2^-23 of it and fl(x / s) by 2^-24, so
// for quotients below 7.5 the two are within 1.4e-6: both round to one integer where the
// product is further than 5e-6 from halfway between two. (A NaN r is answered false.)
__host__ __device__ __forceinline__ bool code8_clear(float x, float r, uint32_t &c) {
  const float q = mul_rn(x, r), y = add_rn(q, 12582920.0f);
  c = bits_of(y);
  return fabsf(add_rn(q, -add_rn(y, -12582920.0f))) < 0.499995f;
}

__host__ __device__ __forceinline__ uint64_t pair64(float lo, float hi) {
#ifdef __CUDA_ARCH__
  uint64_t x;
  asm("mov.b64 %0, {%1, %2};" : "=l"(x) : "f"(lo), "f"(hi));
  return x;
#else
  return static_cast<uint64_t>(bits_of(hi)) << 32 | bits_of(lo);
#endif
}

// code + 8 in bits 0-3, of two floats given by their bits, in their places; each has its own
// scale, ns = (-s_lo, -s_hi) and r = (r_lo, r_hi) as pair64. On the device the four operations
// run on both at once as packed f32x2 instructions (per half the same IEEE operations).
// Bits 4-7 are zero but for a NaN, whose sum has every bit set.
__host__ __device__ __forceinline__ void code8_pair(uint32_t &lo, uint32_t &hi, uint64_t ns,
                                                    uint64_t r) {
#ifdef __CUDA_ARCH__
  uint64_t x, q0, e, q, y;
  asm("mov.b64 %0, {%1, %2};" : "=l"(x) : "r"(lo), "r"(hi));
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(q0) : "l"(x), "l"(r));
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(e) : "l"(q0), "l"(ns), "l"(x));
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(q) : "l"(e), "l"(r), "l"(q0));
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(y) : "l"(q), "l"(0x4B4000084B400008ull));
  asm("mov.b64 {%0, %1}, %2;" : "=r"(lo), "=r"(hi) : "l"(y));
#else
  const auto sum = [](uint32_t x, uint32_t s, uint32_t i) {
    float f[3];
    const uint32_t u[3] = {x, s ^ 0x80000000u, i};
    memcpy(f, u, 12);
    const uint32_t y = code8_recip(f[0], f[1], f[2]);
    return (y & 0x7fffffffu) > 0x7f800000u ? 0x7fffffffu : y;  // the device's NaN
  };
  lo = sum(lo, static_cast<uint32_t>(ns), static_cast<uint32_t>(r));
  hi = sum(hi, static_cast<uint32_t>(ns >> 32), static_cast<uint32_t>(r >> 32));
#endif
}

// One code byte of them, in bits 0-7 of the result, lo in the low nibble.
__host__ __device__ __forceinline__ uint32_t code_byte_pair(uint32_t lo, uint32_t hi, uint64_t ns,
                                                            uint64_t r) {
  code8_pair(lo, hi, ns, r);
  return hi * 16u + (lo & 15u);  // (a NaN in lo would borrow from the high nibble)
}

}  // namespace kvq
