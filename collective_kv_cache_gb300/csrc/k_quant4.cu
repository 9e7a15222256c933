// k_quant4.cu - 4-bit pages: tokens' K and V quantised into their slots, and slots read back.
//
// int4, a head row x of D elements: s = the least bf16 >= (hi - lo) / 15 (hi = max(0, max x), lo =
// min(0, min x)), z = rne(-lo / s), code = clamp(rne(x / s) + z, 0, 15). "The least bf16" is decided by
// 15 s - hi >= -lo with the left side rounded down in one fma, which is exact as a comparison;
// nearest quotients by the exact residual x - n s, as the 8-bit pages' (k_quant.cu).
// e2m1, a quarter of a row: s = the least power of two with amax <= 6 s, so x / s is exact, and the
// conversion instruction rounds it to the nearest code.
// Reading back: bf16((code - z) s), or code * s, which is a bf16 (and NaN in a quarter whose byte is 255).
//
// Both kernels move 2.53 bytes an element once (D = 128). A lane of the write takes 16 elements (32
// bytes in, 8 out), of int4's, which costs more a row, 32; of the read two vectors of 8, half a row
// apart (whole lines stored). A row's extrema are a few shuffles. A CTA takes up to 32 tokens of one
// layer's K or V.
//
// Measured on one GB300 at D = 128: 51200 tokens of 8 layers and 8 heads read back in 314 us from
// either (6.8 TB/s, the rate of a copy; one vector a lane 318 from int4, 330 from e2m1). 7070 tokens of
// 28 layers and 4 heads written and read back in 157 us as e2m1 (5.9 TB/s) and in 172 as int4, whose
// write takes 99 of them, bound by its instructions (issue slots busy in three cycles of four). A
// token of ten agents: 5 us in a graph, the launches.
#include "td_cache4.cuh"

namespace td {

namespace {

// Threads of a CTA; int4's rows have half the lanes of e2m1's in the write (256: 179 us for the
// prompts below written and read, 173 so).
TD_HD constexpr int slot_threads(int kind, bool write) { return write && kind == kCacheInt4 ? 128 : 256; }
constexpr uint32_t kScaleMin = 27u << 23;        // 2^-100

// Page and slot of the CTA's tokens: {-1, 0} skipped, {-2, 0} none of the pool's.
__device__ __forceinline__ int2 place_of(const SlotArgs& A, int t) {
  const int slot = A.slots[t];
  if (slot == -1) return make_int2(-1, 0);
  const PoolDev& p = A.cache.pool;
  const int page = p.p_shift >= 0 ? (slot >> p.p_shift) : slot / p.P;
  if (slot < 0 || page >= p.num_pages) {
    atomicOr(A.err, err_bit(TD_ERR_UNMAPPED_PAGE));
    return make_int2(-2, 0);
  }
  return make_int2(page, slot - page * p.P);
}

constexpr float kMagic = 12582912.0f;    // 1.5 * 2^23: an integer added to it sits in the low bits

// kMagic + rne(x / s) from kMagic + n with n = rne(x * fl(1/s)), which is at most one step off, next to a
// tie. d = x - n s is exact (a multiple of 2^-19 of s's power of two, at most about s; |x| < 2^-12 s:
// n = 0), so comparing it with s / 2 decides; a tie goes to the even one.
__device__ __forceinline__ float settled(float tm, float d, float half) {
  if (fabsf(d) >= half) {
    const bool odd = (__float_as_uint(tm) & 1u) != 0;
    if (fabsf(d) > half || odd) tm = __fadd_rn(tm, copysignf(1.0f, d));
  }
  return tm;
}

// The scale and zero point of a row: hi and -lo as bf16 patterns (finite).
__device__ __forceinline__ uint32_t int4_word(uint32_t hi_bits, uint32_t nlo_bits) {
  const float hi = __uint_as_float(hi_bits << 16), nlo = __uint_as_float(nlo_bits << 16);
  // near (hi - lo) / 15, within a few 2^-24 (sixteenths: the sum stays finite)
  const float about = __fmul_rn(__fadd_rn(hi * 0.0625f, nlo * 0.0625f), 1.06666667f);
  uint32_t bits = __float_as_uint(about) & 0xFFFF0000u;
#pragma unroll
  for (int i = 0; i < 2; ++i)
    if (!(__fmaf_rd(15.0f, __uint_as_float(bits), -hi) >= nlo)) bits += 0x10000u;
  bits = max(bits, kScaleMin);
  const float s = __uint_as_float(bits);
  const float tm = __fmaf_rn(nlo, __frcp_rn(s), kMagic);
  const float z = settled(tm, __fmaf_rn(-__fadd_rn(tm, -kMagic), s, nlo), 0.5f * s);
  return bits | min(__float_as_uint(z) & 0xFFu, 15u);
}

// Eight codes of a row. rne(x / s) + zero is 0 or more, since -zero is the least quotient rounded, but
// can pass 15 by one: x is taken as `most` at most, a bf16 whose quotient rounds to 15 - zero.
__device__ __forceinline__ uint32_t int4_codes8(const uint4& v, uint32_t most2, float r, float s,
                                                float half, float zero) {
  uint4 w;
  asm("min.bf16x2 %0, %1, %2;" : "=r"(w.x) : "r"(v.x), "r"(most2));
  asm("min.bf16x2 %0, %1, %2;" : "=r"(w.y) : "r"(v.y), "r"(most2));
  asm("min.bf16x2 %0, %1, %2;" : "=r"(w.z) : "r"(v.z), "r"(most2));
  asm("min.bf16x2 %0, %1, %2;" : "=r"(w.w) : "r"(v.w), "r"(most2));
  float x[8], tm[8], d[8], far = 0.0f;
  unpack8(w, x);
  const float2 r2 = make_float2(r, r), s2 = make_float2(-s, -s), up = make_float2(kMagic, kMagic);
#pragma unroll
  for (int i = 0; i < 8; i += 2) {
    const float2 x2 = make_float2(x[i], x[i + 1]);
    const float2 t2 = fma2(x2, r2, up), d2 = fma2(add2(t2, make_float2(-kMagic, -kMagic)), s2, x2);
    tm[i] = t2.x;
    tm[i + 1] = t2.y;
    d[i] = d2.x;
    d[i + 1] = d2.y;
    far = max3(far, fabsf(d2.x), fabsf(d2.y));
  }
  if (far >= half) {                    // (one next to a tie: seldom)
#pragma unroll
    for (int i = 0; i < 8; ++i) tm[i] = settled(tm[i], d[i], half);
  }
  // sixteen times the sum so far and the next one's bits: kMagic's own bits add up to a constant
  uint32_t sum = 0u, extra = 0u;
#pragma unroll
  for (int i = 6; i >= 0; i -= 2) {
    const float2 c = add2(make_float2(tm[i], tm[i + 1]), make_float2(zero, zero));
    sum = (sum * 16u + __float_as_uint(c.y)) * 16u + __float_as_uint(c.x);
    extra = (extra * 16u + 0x4B400000u) * 16u + 0x4B400000u;
  }
  return sum - extra;
}

// Biased exponent of the least power of two with amax <= 6 of it (top: amax's bf16 pattern).
__device__ __forceinline__ uint32_t e2m1_byte(uint32_t top) {
  // amax = m 2^e: e - 2 for m <= 1.5 (6 = 1.5 * 2^2), else e - 1; adding just under a half to the
  // fraction carries exactly when m > 1.5
  const int b = static_cast<int>(((top << 16) + 0x003FFFFFu) >> 23) - 2;
  return static_cast<uint32_t>(max(b, 27));
}

__device__ __forceinline__ uint32_t e2m1_codes8(const float* x, uint32_t byte) {
  const float r = __uint_as_float((254u - byte) << 23);      // a power of two: x * r is exact
  uint32_t y;
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, d};\n\t}"
      : "=r"(y)
      : "f"(x[0] * r), "f"(x[1] * r), "f"(x[2] * r), "f"(x[3] * r), "f"(x[4] * r), "f"(x[5] * r),
        "f"(x[6] * r), "f"(x[7] * r));
  return y;
}

// Of 8 bf16, the larger halves as signed 16-bit numbers (positive values in order, over the negative
// ones), and as unsigned ones (negative values by magnitude, over the positive ones).
__device__ __forceinline__ uint32_t highest8(const uint4& v) {
  return __vmaxs2(__vmaxs2(v.x, v.y), __vmaxs2(v.z, v.w));
}
__device__ __forceinline__ uint32_t lowest8(const uint4& v) {
  return __vmaxu2(__vmaxu2(v.x, v.y), __vmaxu2(v.z, v.w));
}
__device__ __forceinline__ uint32_t magnitudes8(const uint4& v) {
  return __vmaxu2(__vmaxu2(v.x & 0x7FFF7FFFu, v.y & 0x7FFF7FFFu),
                  __vmaxu2(v.z & 0x7FFF7FFFu, v.w & 0x7FFF7FFFu));
}

// Eight codes' values as bf16.
template <int kKind>
__device__ __forceinline__ uint4 values8(uint32_t c, uint32_t word, int quarter) {
  if constexpr (kKind == kCacheInt4) {
    // code - zero is a bf16 (128 + code less 128 + zero), and its product with the scale is rounded once
    const uint32_t z = 0x4300u | (word & 0xFu), z2 = z | (z << 16), s2 = __byte_perm(word, 0u, 0x3232);
    const uint32_t even = c, odd = c >> 4;
    auto two = [&](uint32_t pair) {
      uint32_t d;
      asm("{\n\t.reg .b32 t;\n\tsub.rn.bf16x2 t, %1, %2;\n\tmul.rn.bf16x2 %0, t, %3;\n\t}"
          : "=r"(d) : "r"((pair & 0x000F000Fu) | 0x43004300u), "r"(z2), "r"(s2));
      return d;
    };
    return make_uint4(two(__byte_perm(even, odd, 0x4400)), two(__byte_perm(even, odd, 0x5511)),
                      two(__byte_perm(even, odd, 0x6622)), two(__byte_perm(even, odd, 0x7733)));
  } else {
    const float s = byte_scale((word >> (8 * quarter)) & 0xFFu);
    const uint32_t h[4] = {e2m1_f16<0>(c), e2m1_f16<1>(c), e2m1_f16<2>(c), e2m1_f16<3>(c)};
    uint32_t y[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) y[i] = pack_bf2(__fmul_rn(f16_lo(h[i]), s), __fmul_rn(f16_hi(h[i]), s));
    return make_uint4(y[0], y[1], y[2], y[3]);
  }
}

}  // namespace

// A CTA: per_cta tokens of one layer's K or V. A thread's vectors are kThreads apart, so their
// (token, head) advance by a fixed step.
template <int D, int kKind, bool kWrite>
__global__ void __launch_bounds__(slot_threads(kKind, kWrite))
slots_kernel(const __grid_constant__ SlotArgs A) {
  constexpr int kThreads = slot_threads(kKind, kWrite);
  constexpr int kPer = kWrite && kKind == kCacheInt4 ? 32 : 16;   // elements per lane
  constexpr int kIn = kPer / 8;                        // 16-byte vectors of them
  constexpr int kLanes = D / kPer;                     // lanes per head row
  // rows in flight per thread (e2m1's write: two 165 us, int4's: one 189, four 191)
  constexpr int kUnroll = !kWrite ? 4 : (kKind == kCacheInt4 ? 2 : 1);
  __shared__ int2 s_place[kQuantTokens];
  pdl_wait();
  const int t0 = blockIdx.x * A.per_cta, nt = min(A.per_cta, A.n - t0);
  if (static_cast<int>(threadIdx.x) < nt) s_place[threadIdx.x] = place_of(A, t0 + threadIdx.x);
  __syncthreads();
  pdl_trigger();
  const int li = blockIdx.y >> 1, kv = blockIdx.y & 1;
  const PoolDev& pool = A.cache.pool;
  const int H = A.g.H, P = pool.P;
  const int64_t plane =
      (static_cast<int64_t>(A.layer_begin + li) * 2 + kv) * pool.num_pages * H * P;
  uint8_t* codes = reinterpret_cast<uint8_t*>(pool.base) + plane * (D / 2);
  uint32_t* words = A.cache.word + plane;
  uint16_t* dense = (kv ? A.v : A.k) + (static_cast<int64_t>(li) * A.n + t0) * A.g.E;
  const int rows = nt * H;                             // head rows of the CTA
  // a lane's vectors: side by side in the write, in the read half a row apart (whole lines stored)
  const int part = threadIdx.x % kLanes;
  int r = threadIdx.x / kLanes;
  int tok = static_cast<int>((static_cast<uint32_t>(r) * A.head_mul) >> 20);
  int h = r - tok * H;
  constexpr int kStep = kThreads / kLanes;
  const int step_tok = static_cast<int>((static_cast<uint32_t>(kStep) * A.head_mul) >> 20);
  const int step_h = kStep - step_tok * H;
  // (as many rounds for every thread: the shuffles below are the whole warp's)
  for (int first = 0; first < rows; first += kStep * kUnroll) {
    int row[kUnroll], rr[kUnroll];        // head row in the plane; -1 skipped, -2 not the pool's
    uint4 x[kUnroll][kIn];
    uint32_t cw[kUnroll][kIn], wd[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      row[u] = -1;
      rr[u] = r;
#pragma unroll
      for (int i = 0; i < kIn; ++i) {
        x[u][i] = make_uint4(0u, 0u, 0u, 0u);
        cw[u][i] = 0u;
      }
      wd[u] = 0u;
      if (r < rows) {
        const int2 at = s_place[tok];
        row[u] = at.x < 0 ? at.x : (at.x * H + h) * P + at.y;
      }
      if constexpr (kWrite) {
        if (row[u] >= 0) {
#pragma unroll
          for (int i = 0; i < kIn; ++i)
            x[u][i] = ldg16(dense + static_cast<int64_t>(r) * D + part * kPer + i * 8);
        }
      } else if (row[u] >= 0) {
        const uint32_t* from = reinterpret_cast<const uint32_t*>(codes + static_cast<int64_t>(row[u]) * (D / 2));
#pragma unroll
        for (int i = 0; i < kIn; ++i) cw[u][i] = __ldg(from + part + i * kLanes);
        wd[u] = __ldg(words + row[u]);
      }
      r += kStep;
      tok += step_tok;
      h += step_h;
      if (h >= H) {
        h -= H;
        ++tok;
      }
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      if constexpr (kWrite) {
        uint32_t word;
        bool finite;
        uint32_t c[kIn];
        if constexpr (kKind == kCacheInt4) {
          uint32_t up = highest8(x[u][0]), dn = lowest8(x[u][0]);
#pragma unroll
          for (int i = 1; i < kIn; ++i) {
            up = __vmaxs2(up, highest8(x[u][i]));
            dn = __vmaxu2(dn, lowest8(x[u][i]));
          }
          // the lane's highest in the low half, its lowest's negative in the high half
          uint32_t lows = max(dn & 0xFFFFu, dn >> 16) ^ 0x8000u;
          if (lows & 0x8000u) lows = 0u;            // (none is negative)
          uint32_t m = __vmaxs2(__vmaxs2(up, __byte_perm(up, 0u, 0x1032)), 0u);
          m = (m & 0xFFFFu) | (lows << 16);
#pragma unroll
          for (int o = kLanes / 2; o > 0; o >>= 1)
            m = __vmaxu2(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
          const uint32_t hi = m & 0xFFFFu, nlo = m >> 16;
          finite = hi < 0x7F80u && nlo < 0x7F80u;
          word = finite ? int4_word(hi, nlo) : 0x7FC00000u;
          const float s = __uint_as_float(word & 0xFFFF0000u);
          const float zero = static_cast<float>(word & 0xFFFFu);
          // (15.25 - zero) s cut to a bf16: less than 2^-7 of it, 0.12 s, below
          const uint32_t most = __float_as_uint((15.25f - zero) * s);
          const uint32_t most2 = __byte_perm(most, 0u, 0x3232);
          const float r1 = __frcp_rn(s), half = 0.5f * s;
#pragma unroll
          for (int i = 0; i < kIn; ++i) c[i] = int4_codes8(x[u][i], most2, r1, s, half, zero);
        } else {
          uint32_t m = __vmaxu2(magnitudes8(x[u][0]), magnitudes8(x[u][1]));
          if constexpr (D == 128) m = __vmaxu2(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
          const uint32_t top = max(m & 0xFFFFu, m >> 16);
          const uint32_t byte = e2m1_byte(top);
          // a quarter is kLanes / 4 lanes: its byte in its place, then all four together
          constexpr int kQuarter = kLanes / 4;
          word = top < 0x7F80u ? byte << (8 * (part / kQuarter)) : 0xFFFFFFFFu;
#pragma unroll
          for (int o = kQuarter; o < kLanes; o *= 2) word |= __shfl_xor_sync(0xFFFFFFFFu, word, o);
          finite = word != 0xFFFFFFFFu;
#pragma unroll
          for (int i = 0; i < kIn; ++i) {
            float f[8];
            unpack8(x[u][i], f);
            c[i] = e2m1_codes8(f, byte);
          }
        }
        if (row[u] < 0) continue;
        if (!finite) {                    // the row reads back as NaN
#pragma unroll
          for (int i = 0; i < kIn; ++i) c[i] = 0u;
          if (part == 0) atomicOr(A.err, err_bit(TD_ERR_NONFINITE));
        }
        uint8_t* to = codes + static_cast<int64_t>(row[u]) * (D / 2) + part * (kPer / 2);
        if constexpr (kIn == 4) *reinterpret_cast<uint4*>(to) = make_uint4(c[0], c[1], c[2], c[3]);
        else *reinterpret_cast<uint2*>(to) = make_uint2(c[0], c[kIn - 1]);
        if (part == 0) words[row[u]] = word;
      } else {
        if (row[u] == -1) continue;
        uint16_t* to = dense + static_cast<int64_t>(rr[u]) * D + part * 8;
#pragma unroll
        for (int i = 0; i < kIn; ++i) {
          uint4 out = values8<kKind>(cw[u][i], wd[u], part / (kLanes / 2) + 2 * i);
          if (row[u] == -2) out = make_uint4(0u, 0u, 0u, 0u);
          st16(to + i * kLanes * 8, out);
        }
      }
    }
  }
}

template <bool kWrite>
static cudaError_t run(const SlotArgs& a, CacheKind kind, cudaStream_t st) {
  const dim3 grid((a.n + a.per_cta - 1) / a.per_cta, a.nl * 2);
  const bool wide = a.g.D == 128;
  const int threads = slot_threads(kind, kWrite);
  if (kind == kCacheInt4)
    return wide ? launch_after(slots_kernel<128, kCacheInt4, kWrite>, grid, threads, 0, st, a)
                : launch_after(slots_kernel<64, kCacheInt4, kWrite>, grid, threads, 0, st, a);
  return wide ? launch_after(slots_kernel<128, kCacheE2m1, kWrite>, grid, threads, 0, st, a)
              : launch_after(slots_kernel<64, kCacheE2m1, kWrite>, grid, threads, 0, st, a);
}

cudaError_t launch_quantise4(const SlotArgs& a, CacheKind kind, cudaStream_t st) {
  return run<true>(a, kind, st);
}
cudaError_t launch_dequantise4(const SlotArgs& a, CacheKind kind, cudaStream_t st) {
  return run<false>(a, kind, st);
}

}  // namespace td
