// The 4-bit row format of include/snapkv_cache.h: words of eight levels, and how they become operands.
//
// A 16-bit half of a word holds the levels of four channels as [s0 s1 m2 m3 | s2 s3 m0 m1] (one bit
// per sign s, three per m = (|t| - 1) / 2). With the sign moved to bit 15 and m above one constant
// low bit, the half is a subnormal bf16: +-(2m + 1) = t in units of 2^-131 (pairs 0 and 2) or 2^-133
// (pairs 1 and 3). mma.sync takes subnormal bf16 operands exactly, so levels become operands with one
// AND-OR per two channels and no conversion, subtraction or table (measured on a GB300: products with
// such operands are exact); the powers of two are undone where they cost nothing.
#pragma once

#include "snapkv_common.cuh"

namespace snapkv {

constexpr int kQ4Group = 64;   // channels that share one (h, z)

constexpr uint32_t kQ4MaskEven = 0x80388038u, kQ4OneEven = 0x00040004u;   // pairs 0, 2: t * 2^-131
constexpr uint32_t kQ4MaskOdd = 0x800E800Eu, kQ4OneOdd = 0x00010001u;     // pairs 1, 3: t * 2^-133

__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t sel) { return __byte_perm(a, b, sel); }

// The constant bits, as a kernel argument: an AND-OR takes one immediate at most, and with both constants
// known to the compiler it becomes two instructions.
struct Q4Ones {
  uint32_t even = kQ4OneEven, odd = kQ4OneOdd;
};

// The operands of pairs 0 .. 3 from a register with the two halves as stored (w) and with each
// half's bytes swapped (s).
__device__ __forceinline__ void q4_operands(const Q4Ones& one, uint32_t w, uint32_t s, uint32_t* out) {
  out[0] = (w & kQ4MaskEven) | one.even;
  out[1] = ((w << 1) & kQ4MaskOdd) | one.odd;
  out[2] = (s & kQ4MaskEven) | one.even;
  out[3] = ((s << 1) & kQ4MaskOdd) | one.odd;
}

// Two fp32 operations in one instruction (each rounded as usual).
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 r;
  asm("add.rn.f32x2 %0, %1, %2;"
      : "=l"(reinterpret_cast<uint64_t&>(r))
      : "l"(reinterpret_cast<uint64_t&>(a)), "l"(reinterpret_cast<uint64_t&>(b)));
  return r;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;"
      : "=l"(reinterpret_cast<uint64_t&>(r))
      : "l"(reinterpret_cast<uint64_t&>(a)), "l"(reinterpret_cast<uint64_t&>(b)), "l"(reinterpret_cast<uint64_t&>(c)));
  return r;
}

__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 r;
  asm("mul.rn.f32x2 %0, %1, %2;"
      : "=l"(reinterpret_cast<uint64_t&>(r))
      : "l"(reinterpret_cast<uint64_t&>(a)), "l"(reinterpret_cast<uint64_t&>(b)));
  return r;
}

// Word index, within a row of NG groups, of channels 8 * o .. 8 * o + 7 of group g.
template <int NG> __device__ __forceinline__ constexpr int q4_word(int g, int o) { return NG * o + g; }

// Packs eight level numbers u of channels 0 .. 7, given as nibbles in the order (from bit 0 up)
// 2 0 6 4 3 1 7 5, into a word. In that order each half has its pairs' nibbles as [2 3 | 0 1], so that two
// of the four m fields are in place and two are one bit off, and the signs are a byte swap away.
__device__ __forceinline__ uint32_t q4_pack(uint32_t x) {
  const uint32_t neg = ~x & 0x88888888u;                               // u < 8: t negative
  const uint32_t mag = (x ^ (neg - (neg >> 3))) & 0x77777777u;         // u - 8, or 7 - u
  const uint32_t s = prmt(neg, neg, 0x2301);
  return (mag & 0x07070707u) | ((mag >> 1) & 0x38383838u) | (s & 0x80808080u) | ((s << 3) & 0x40404040u);
}

}  // namespace snapkv
