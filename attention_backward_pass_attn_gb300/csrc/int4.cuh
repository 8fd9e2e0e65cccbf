// int4.cuh -- rows of 4-bit values, as the 4-bit key/value cache holds them.
//
// 32 neighbouring values of a row share a factor f, a bf16 number of five
// significant bits; a value is c f with c in -7 .. 7, held as the four bits of
// c + 8, element 2i of a row in the low half of byte i and 2i + 1 in the high
// half.  c has three bits and f five, so c f is a bf16 number: what the cache
// stands for is known to the last bit, and meets the tensor core unrounded.
#pragma once

#include <stdint.h>

#include "ptx.cuh"

namespace attn {

constexpr int kInt4Group = 32;  // values that share a factor

// Nibbles p and p + 4 of a word (p = 0 .. 3) as two bf16 values, times f (two
// bf16 factors).  128 + n is a bf16 number whose last bits are the nibble n:
// 136 off it is c, exactly, in one addition.
__device__ __forceinline__ uint32_t int4_pair(uint32_t w, int p, uint32_t f) {
  uint32_t x = w >> (4 * p);
  // a & b | c, said in one instruction: written out in C it took two, a sixth
  // of the single-token attention's
  asm("lop3.b32 %0, %0, %1, %2, 0xEA;" : "+r"(x) : "r"(0x000F000Fu), "r"(0x43004300u));
  asm("add.rn.bf16x2 %0, %1, %2;" : "=r"(x) : "r"(x), "r"(0xC308C308u));
  return mul_bf16x2(x, f);
}

// The same in an instruction less, for factors f below 2^123: with the nibble
// four bits below a bf16 number's leading one, 16 + n, the 24 to take off is a
// number of two bits, and 24 f still one of bf16's eight: (16 + n) f - 24 f is
// c f, exactly, in one multiply-add.
__device__ __forceinline__ uint32_t int4_off(uint32_t f) {  // -24 f
  return mul_bf16x2(f, 0xC1C0C1C0u);
}
__device__ __forceinline__ uint32_t int4_pair(uint32_t w, int p, uint32_t f, uint32_t off) {
  uint32_t x = p == 0 ? w << 3 : w >> (4 * p - 3);
  asm("lop3.b32 %0, %0, %1, %2, 0xEA;" : "+r"(x) : "r"(0x00780078u), "r"(0x41804180u));
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(x) : "r"(x), "r"(f), "r"(off));
  return x;
}

}  // namespace attn
