// Decode of 8-bit activation codes (act8.cu), shared by the restore kernel and
// the adapter-gradient kernel that reads a checkpoint.
#pragma once

#include "common.cuh"

namespace qlora {

__device__ __forceinline__ uint32_t sub_bf16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

// Four int8 codes of one word -> four bf16 values q * sc, in order; s2 holds
// the block's bf16 scale in both halves.  q is formed exactly: with the byte
// in two's complement, q = (128 + (b & 127)) - (128 + (b & 128)), and both
// terms are bf16 bit patterns (0x4300 is 128, 0x4380 is 256).  The product is
// rounded once to bf16, as X^ is defined.
__device__ __forceinline__ void act8_decode4(uint32_t w, uint32_t s2, uint32_t &lo, uint32_t &hi) {
  const uint32_t a = prmt(w, 0u, 0x4140), b = prmt(w, 0u, 0x4342);   // one byte per half word
  const uint32_t qa = sub_bf16x2((a & 0x007F007Fu) | 0x43004300u, (a & 0x00800080u) | 0x43004300u);
  const uint32_t qb = sub_bf16x2((b & 0x007F007Fu) | 0x43004300u, (b & 0x00800080u) | 0x43004300u);
  lo = mul_bf16x2(qa, s2);
  hi = mul_bf16x2(qb, s2);
}

}  // namespace qlora
