// k_quant.cu - 8-bit pages: new tokens' K and V quantised as they are written, and read back.
//
// One scale per head row (position, kv head) of D elements x:
//   int8   s = max(fl32(amax / 127), 2^-100),        code = rne(x / s)
//   e4m3   s = max(2^ceil(log2(amax / 448)), 2^-100), code = rne_e4m3(x / s)
// The quotient is the real one: no code depends on how a division is rounded. e4m3 keeps its
// relative precision under any scale, so its scale is a power of two and x / s is exact; int8
// steps are uniform, so its scale uses the whole range and the nearest code is decided by the
// exact residual x - n s (below). Reading back: bf16(fl32(code * s)).
//
// Both kernels move 2 + 1 + 4/D bytes an element once and are bound by HBM. A group of lanes
// (D / 8, rounded up to a power of two) holds one head row, 8 elements a lane in one 16-byte
// vector, so the row's maximum is a few shuffles and no row is read twice. A CTA takes up to
// 32 tokens of one layer and K or V; their page rows are looked up once, by one thread each.
#include "td_device.cuh"

namespace td {

namespace {

constexpr int kThreads = 256;
constexpr int kUnroll = 4;   // vectors in flight per thread
constexpr float kScaleMin = 7.8886090522101181e-31f;   // 2^-100: keeps 1 / s finite

// Row (page * P + slot) of the launch's token t, or -1 and the error bit.
__device__ __forceinline__ int token_row(const ChunkList& list, const PoolDev& p, int t,
                                         uint32_t* err) {
  int lo = 0, hi = list.n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (list.row[mid] <= t) lo = mid;
    else hi = mid - 1;
  }
  const int pos = list.start[lo] + t - list.row[lo];
  const int lp = p.p_shift >= 0 ? (pos >> p.p_shift) : pos / p.P;
  int32_t page = -1;
  if (lp < p.max_lp) page = __ldg(p.bt + static_cast<int64_t>(list.agent[lo]) * p.max_lp + lp);
  if (page < 0 || page >= p.num_pages) {
    atomicOr(err, err_bit(TD_ERR_UNMAPPED_PAGE));
    return -1;
  }
  return page * p.P + (pos - lp * p.P);
}

// Scale of a row whose largest magnitude is the bf16 pattern `top` (finite).
template <int kKind>
__device__ __forceinline__ float row_scale(uint32_t top) {
  if constexpr (kKind == kCacheInt8) {
    return fmaxf(__fdiv_rn(__uint_as_float(top << 16), 127.0f), kScaleMin);
  } else {
    // amax = m 2^e: exponent e - 8 for m <= 1.75 (448 = 1.75 * 2^8), else e - 7; adding
    // just under a quarter to the fraction carries exactly when m > 1.75
    const int ex = static_cast<int>(((top << 16) + 0x001FFFFFu) >> 23) - 8;
    return __uint_as_float(static_cast<uint32_t>(max(ex, 27)) << 23);
  }
}

// The int8 code of x: n = rne(x * fl(1/s)) is at most one step off, and only where x / s is
// next to a tie. d = x - n s is exact: it is a multiple of ulp(s) (x is a bf16, so it is one
// too unless |x| < 2^-15 s, where n = 0) and at most about s, so one fma gives it unrounded
// and comparing it with s / 2 places x on the right side; a tie goes to the even code.
__device__ __forceinline__ uint32_t int8_code(float x, float r, float s, float half) {
  constexpr float kMagic = 12582912.0f;   // 1.5 * 2^23: the integer sits in the low bits
  float tm = __fmaf_rn(x, r, kMagic);
  const float n = __fadd_rn(tm, -kMagic);
  const float d = __fmaf_rn(-n, s, x);
  if (fabsf(d) >= half) {
    const bool odd = (__float_as_uint(tm) & 1u) != 0;
    if (fabsf(d) > half || odd) tm = __fadd_rn(tm, copysignf(1.0f, d));
  }
  return __float_as_uint(tm) & 0xFFu;
}

__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

template <int kKind>
__device__ __forceinline__ uint2 codes8(const float* x, float s) {
  const float r = __frcp_rn(s);
  uint2 c;
  if constexpr (kKind == kCacheInt8) {
    const float half = 0.5f * s;
    uint32_t b[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) b[i] = int8_code(x[i], r, s, half);
    c.x = b[0] | (b[1] << 8) | (b[2] << 16) | (b[3] << 24);
    c.y = b[4] | (b[5] << 8) | (b[6] << 16) | (b[7] << 24);
  } else {
    // s is a power of two: x * (1 / s) is exact, and 448 is the largest value
    c.x = e4m3x2(x[0] * r, x[1] * r) | (e4m3x2(x[2] * r, x[3] * r) << 16);
    c.y = e4m3x2(x[4] * r, x[5] * r) | (e4m3x2(x[6] * r, x[7] * r) << 16);
  }
  return c;
}

// Codes of one 32-bit word as floats.
template <int kKind>
__device__ __forceinline__ void values4(uint32_t w, float* y) {
  if constexpr (kKind == kCacheInt8) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      y[i] = static_cast<float>(static_cast<int8_t>((w >> (8 * i)) & 0xFFu));
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      // sign, exponent and fraction moved to a float's places, 2^120 too small (bias 7
      // against 127); the product is exact, subnormal codes included
      const uint32_t b = (w >> (8 * i)) & 0xFFu;
      y[i] = __fmul_rn(__uint_as_float(((b & 0x80u) << 24) | ((b & 0x7Fu) << 20)), 0x1p120f);
    }
  }
}

}  // namespace

template <int kKind, bool kWrite>
__global__ void __launch_bounds__(kThreads)
quant_kernel(const __grid_constant__ QuantArgs A, const __grid_constant__ ChunkList list) {
  pdl_wait();
  __shared__ int s_row[kQuantTokens];
  const int t0 = blockIdx.x * A.per_cta;
  const int nt = min(A.per_cta, list.row[list.n] - t0);
  if (static_cast<int>(threadIdx.x) < nt)
    s_row[threadIdx.x] = token_row(list, A.cache.pool, t0 + threadIdx.x, A.err);
  __syncthreads();
  const int li = blockIdx.y >> 1, kv = blockIdx.y & 1;
  const int H = A.g.H, D = A.g.D;
  // head rows of this layer and K or V in the pages; this CTA's first dense row
  const int64_t plane = (static_cast<int64_t>(A.layer_begin + li) * 2 + kv) *
                        A.cache.pool.num_pages * A.cache.pool.P * H;
  uint8_t* codes = reinterpret_cast<uint8_t*>(A.cache.pool.base) + plane * D;
  float* scale = A.cache.scale + plane;
  uint16_t* dense = (kv ? A.v : A.k) + (static_cast<int64_t>(li) * A.tokens + A.tok0 + t0) * A.g.E;
  const int lanes = 1 << A.lane_shift;
  const int total = nt * H << A.lane_shift;
  for (int base = 0; base < total; base += kThreads * kUnroll) {
    int64_t at[kUnroll];     // head row in the pages, -1: nothing to do
    int src[kUnroll];        // element offset of the vector from the CTA's first dense row
    int e0[kUnroll];         // element offset within the head row
    uint4 x[kUnroll];
    uint2 cw[kUnroll];
    float sc[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int i = base + u * kThreads + threadIdx.x;
      e0[u] = (i & (lanes - 1)) * 8;
      at[u] = -1;
      src[u] = 0;
      x[u] = make_uint4(0u, 0u, 0u, 0u);
      cw[u] = make_uint2(0u, 0u);
      sc[u] = 0.0f;
      if (i >= total || e0[u] >= D) continue;
      const int r = i >> A.lane_shift;
      const int tok = static_cast<int>((static_cast<uint32_t>(r) * A.head_mul) >> 20);
      const int h = r - tok * H;
      src[u] = r * D + e0[u];
      const int row = s_row[tok];
      at[u] = row < 0 ? -1 : static_cast<int64_t>(row) * H + h;
      if constexpr (kWrite) {
        x[u] = ldg16(dense + src[u]);
      } else if (row >= 0) {
        cw[u] = __ldg(reinterpret_cast<const uint2*>(codes + at[u] * D + e0[u]));
        sc[u] = __ldg(scale + at[u]);
      }
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int i = base + u * kThreads + threadIdx.x;
      if constexpr (kWrite) {
        uint32_t m = __vmaxu2(__vmaxu2(x[u].x & 0x7FFF7FFFu, x[u].y & 0x7FFF7FFFu),
                              __vmaxu2(x[u].z & 0x7FFF7FFFu, x[u].w & 0x7FFF7FFFu));
        for (int o = lanes >> 1; o > 0; o >>= 1) m = __vmaxu2(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
        const uint32_t top = max(m & 0xFFFFu, m >> 16);
        if (at[u] < 0) continue;
        float s = row_scale<kKind>(top);
        uint2 c = make_uint2(0u, 0u);
        if (top < 0x7F80u) {
          float f[8];
          unpack8(x[u], f);
          c = codes8<kKind>(f, s);
        } else {             // a NaN or an infinity: the row reads back as NaN
          s = __uint_as_float(0x7FC00000u);
          if (e0[u] == 0) atomicOr(A.err, err_bit(TD_ERR_NONFINITE));
        }
        *reinterpret_cast<uint2*>(codes + at[u] * D + e0[u]) = c;
        if (e0[u] == 0) scale[at[u]] = s;
      } else {
        if (i >= total || e0[u] >= D) continue;
        float y[8];          // an unmapped row reads as zeros
        values4<kKind>(cw[u].x, y);
        values4<kKind>(cw[u].y, y + 4);
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] = at[u] < 0 ? 0.0f : __fmul_rn(y[j], sc[u]);
        st16(dense + src[u], pack8(y));
      }
    }
  }
}

template <bool kWrite>
static cudaError_t run(const QuantArgs& a, const ChunkList& list, CacheKind kind,
                       cudaStream_t st) {
  const int tokens = list.row[list.n];
  if (tokens == 0) return cudaSuccess;
  const dim3 grid((tokens + a.per_cta - 1) / a.per_cta, a.nl * 2);
  if (kind == kCacheInt8) return launch_after(quant_kernel<kCacheInt8, kWrite>, grid, kThreads, 0, st, a, list);
  return launch_after(quant_kernel<kCacheE4m3, kWrite>, grid, kThreads, 0, st, a, list);
}

cudaError_t launch_quantise(const QuantArgs& a, const ChunkList& list, CacheKind kind,
                            cudaStream_t st) {
  return run<true>(a, list, kind, st);
}

cudaError_t launch_dequantise(const QuantArgs& a, const ChunkList& list, CacheKind kind,
                              cudaStream_t st) {
  return run<false>(a, list, kind, st);
}

}  // namespace td
