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

// The same times 2^-16, for factors of [2^-110, 2^11), in a mask and a
// multiply-add and half a shift.  A nibble in the lowest or next lowest four bits
// of a bf16 number is, its exponent being 0 or 1, n or 16 n times 2^-133, and with
// a factor 2^117 or 2^113 times the group's one multiply-add makes (n - 8) f 2^-16
// of it, exactly: what it adds has at most nine bits.
constexpr float kInt4Up = 65536.f;
constexpr uint32_t kInt4LowFactor = 0x0880, kInt4Factors = 0x4500 - 0x0880;  // bf16 bits, count
struct Int4Factor {
  uint32_t f;               // two factors, bf16
  uint32_t low, high, off;  // f 2^117, f 2^113, -8 f 2^-16
};
__device__ __forceinline__ Int4Factor int4_factor(uint32_t f) {
  return {f, mul_bf16x2(f, 0x7A007A00u), mul_bf16x2(f, 0x78007800u), mul_bf16x2(f, 0xB900B900u)};
}
__device__ __forceinline__ uint32_t int4_pair_down(uint32_t w, int p, const Int4Factor& f) {
  uint32_t x = (p & 2 ? w >> 8 : w) & (p & 1 ? 0x00F000F0u : 0x000F000Fu);
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(x) : "r"(x), "r"(p & 1 ? f.high : f.low), "r"(f.off));
  return x;
}

}  // namespace attn
