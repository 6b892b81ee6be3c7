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

// The operands of pairs 0 .. 3 from a register with the two halves as stored (w) and with each
// half's bytes swapped (s).
__device__ __forceinline__ void q4_operands(uint32_t w, uint32_t s, uint32_t* out) {
  out[0] = (w & kQ4MaskEven) | kQ4OneEven;
  out[1] = ((w << 1) & kQ4MaskOdd) | kQ4OneOdd;
  out[2] = (s & kQ4MaskEven) | kQ4OneEven;
  out[3] = ((s << 1) & kQ4MaskOdd) | kQ4OneOdd;
}

// Word index, within a row of NG groups, of channels 8 * o .. 8 * o + 7 of group g.
template <int NG> __device__ __forceinline__ constexpr int q4_word(int g, int o) { return NG * o + g; }

// Packs eight level numbers, given as nibbles u of x (channel e in bits 4e .. 4e + 3), into a word.
__device__ __forceinline__ uint32_t q4_pack(uint32_t x) {
  const uint32_t neg = ~x & 0x88888888u;              // u < 8: t negative
  const uint32_t mag = (x ^ ((neg >> 3) * 7u)) & 0x77777777u;   // u - 8, or 7 - u
  uint32_t w = 0;
  constexpr int kSign[4] = {15, 14, 7, 6}, kMag[4] = {3, 0, 11, 8};
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const int at = 16 * (e & 1), j = e >> 1;
    w |= ((neg >> (4 * e + 3)) & 1u) << (at + kSign[j]);
    w |= ((mag >> (4 * e)) & 7u) << (at + kMag[j]);
  }
  return w;
}

// The level of channel e (0 .. 7) of a word.
__device__ __forceinline__ int q4_level(uint32_t w, int e) {
  const uint32_t half = w >> (16 * (e & 1));
  const int j = e >> 1;
  const int sign = j == 0 ? 15 : j == 1 ? 14 : j == 2 ? 7 : 6, at = j == 0 ? 3 : j == 1 ? 0 : j == 2 ? 11 : 8;
  const int t = 2 * (int)((half >> at) & 7u) + 1;
  return (half >> sign) & 1u ? -t : t;
}

}  // namespace snapkv
