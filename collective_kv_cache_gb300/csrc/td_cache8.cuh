// td_cache8.cuh - 8-bit codes as bf16 pairs.
#pragma once

#include "td_device.cuh"

namespace td {

// Two codes, in the high bytes of the halves (kCacheE4m3) or in the low bytes (kCacheInt8),
// as two bf16 of exactly their values; the other bytes may hold anything.
constexpr uint32_t kE4m3Factor = 0x7B807B80u;   // 2^120, twice

template <int kKind>
__device__ __forceinline__ uint32_t codes_bf16(uint32_t u, uint32_t factor = kE4m3Factor) {
  uint32_t y;
  if constexpr (kKind == kCacheE4m3) {
    // exponent and fraction moved to bf16's places: 2^120 too small (bias 7 against 127). The
    // factor may be 2^120 times another power of two: the product stays exact
    asm("mul.rn.bf16x2 %0, %1, %2;"
        : "=r"(y)
        : "r"((u & 0x80008000u) | ((u >> 4) & 0x07F007F0u)), "r"(factor));
  } else {
    // 128 + (low 7 bits) minus 128, or 256 for a negative code: all exact in 8 bits
    asm("sub.rn.bf16x2 %0, %1, %2;"
        : "=r"(y)
        : "r"((u & 0x007F007Fu) | 0x43004300u), "r"((u & 0x00800080u) | 0x43004300u));
  }
  return y;
}

// The codes of a word's bytes 0, 1 (kHigh: 2, 3) as two bf16.
template <int kKind, bool kHigh>
__device__ __forceinline__ uint32_t word_bf16(uint32_t w, uint32_t factor = kE4m3Factor) {
  constexpr uint32_t sel = kKind == kCacheE4m3 ? (kHigh ? 0x3424u : 0x1404u)
                                               : (kHigh ? 0x4342u : 0x4140u);
  return codes_bf16<kKind>(__byte_perm(w, 0u, sel), factor);
}

// Byte i of a and byte i of b as two bf16.
template <int kKind>
__device__ __forceinline__ uint32_t pair_bf16(uint32_t a, uint32_t b, int i) {
  return codes_bf16<kKind>(kKind == kCacheE4m3 ? __byte_perm(a, b, ((4 + i) << 12) | (i << 4))
                                               : __byte_perm(a, b, ((4 + i) << 8) | i));
}

}  // namespace td
