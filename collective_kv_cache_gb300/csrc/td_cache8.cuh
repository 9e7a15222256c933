// td_cache8.cuh - 8-bit codes as pairs of bf16 or f16.
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

// The same as two f16, which hold every code exactly too (e4m3's least value is 2^-9) and cost
// half the instructions. K goes this way, against queries that are scaled row by row
// (f16_scale); V does not, since its other operand is a softmax weight times any scale.
template <int kKind, bool kHigh>
__device__ __forceinline__ uint32_t word_f16(uint32_t w) {
  uint32_t y;
  if constexpr (kKind == kCacheE4m3) {
    if constexpr (kHigh)
      asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, hi;\n\t}"
          : "=r"(y) : "r"(w));
    else
      asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, lo;\n\t}"
          : "=r"(y) : "r"(w));
  } else {
    // 1024 + (code + 128), minus 1152
    asm("sub.rn.f16x2 %0, %1, %2;"
        : "=r"(y)
        : "r"(__byte_perm(w ^ 0x80808080u, 0x64646464u, kHigh ? 0x4342u : 0x4140u)), "r"(0x64806480u));
  }
  return y;
}

// The factor that brings a row whose largest magnitude is the bf16 pattern `top` to [2^14, 2^15),
// and its inverse: powers of two, so that bf16 values become f16 exactly down to 2^-28 of the
// row's largest (smaller ones keep fewer bits, those under 2^-39 of it none).
__device__ __forceinline__ float f16_scale(uint32_t top, float* inverse) {
  const uint32_t e = max(top >> 7, 15u);
  *inverse = __uint_as_float((e - 14u) << 23);
  return __uint_as_float((268u - e) << 23);
}

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// Byte i of a and byte i of b as two bf16.
template <int kKind>
__device__ __forceinline__ uint32_t pair_bf16(uint32_t a, uint32_t b, int i) {
  return codes_bf16<kKind>(kKind == kCacheE4m3 ? __byte_perm(a, b, ((4 + i) << 12) | (i << 4))
                                               : __byte_perm(a, b, ((4 + i) << 8) | i));
}

}  // namespace td
