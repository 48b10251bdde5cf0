// int4 nibbles to fp16 codes without conversions, shared by the kernels that
// feed dequantized tiles to the tensor cores.
#pragma once

#include "kvq_common.cuh"

namespace kvq {

__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t sel) {
  uint32_t d;
  asm("prmt.b32 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(sel));
  return d;
}

__device__ __forceinline__ uint32_t as_u32(__half2 h) { return *reinterpret_cast<uint32_t *>(&h); }
__device__ __forceinline__ __half2 as_h2(uint32_t u) { return *reinterpret_cast<__half2 *>(&u); }

// (w & kMask) | kMagic as one three-input logic op.
template <uint32_t kMask, uint32_t kMagic>
__device__ __forceinline__ uint32_t and_or(uint32_t w) {
  uint32_t d;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(d) : "r"(w), "n"(kMask), "n"(kMagic));
  return d;
}

// Nibbles at bits 0-3 and 16-19 -> fp16 codes: 0x6400 | n is 1024 + n, n = code + 8.
__device__ __forceinline__ uint32_t dq_lo(uint32_t w) {
  const uint32_t x = and_or<0x000F000Fu, 0x64006400u>(w);
  return as_u32(__hsub2(as_h2(x), as_h2(0x64086408u)));  // 1032
}
// Nibbles at bits 4-7 and 20-23: 0x5400 | n << 4 is 64 + n.
__device__ __forceinline__ uint32_t dq_hi(uint32_t w) {
  const uint32_t x = and_or<0x00F000F0u, 0x54005400u>(w);
  return as_u32(__hsub2(as_h2(x), as_h2(0x54805480u)));  // 72
}

__device__ __forceinline__ uint32_t pack_h2(float lo, float hi) {
  return as_u32(__floats2half2_rn(lo, hi));
}
__device__ __forceinline__ float bf_lo(uint32_t u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float bf_hi(uint32_t u) { return __uint_as_float(u & 0xffff0000u); }

}  // namespace kvq
