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
// Both kernels move 2 + 1 + 4/D bytes an element once and are bound by HBM: ten
// chunks of 300 to 1100 tokens, 28 layers of 4 heads, D = 128, are written as e4m3 in 89.5 us,
// and ten of 5120 tokens, 8 layers of 8 heads, read back in 374 us, both at 6.7 to 6.8 TB/s, a
// copy's rate. A call of a few tokens takes 8 us, which are the launch. A group of lanes holds
// one head row, so the row's maximum is a few shuffles and no row is read twice. The
// write takes 16 elements a lane: with 8 the shuffles, scales and addresses cost twice as much
// an element and it ran at 80% of the copy rate, bound by their issue. The read takes 8 (one
// 16-byte store a lane, whole lines a warp): with 16 it ran at 92%. A CTA takes up to
// 32 tokens of one layer and K or V; their page rows are looked up once, by one thread each.
#include "td_cache8.cuh"

namespace td {

namespace {

constexpr int kThreads = 256;
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

// The larger magnitudes of 8 bf16, as bits, by the halves of a word.
__device__ __forceinline__ uint32_t magnitude8(const uint4& v) {
  return __vmaxu2(__vmaxu2(v.x & 0x7FFF7FFFu, v.y & 0x7FFF7FFFu),
                  __vmaxu2(v.z & 0x7FFF7FFFu, v.w & 0x7FFF7FFFu));
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
    // by way of f16, which holds every code exactly, the two NaNs included
    const uint32_t h[2] = {word_f16<kKind, false>(w), word_f16<kKind, true>(w)};
#pragma unroll
    for (int i = 0; i < 2; ++i)
      asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %2;\n\tcvt.f32.f16 %0, lo;\n\t"
          "cvt.f32.f16 %1, hi;\n\t}"
          : "=f"(y[2 * i]), "=f"(y[2 * i + 1]) : "r"(h[i]));
  }
}

}  // namespace

// kShift: log2 of the lanes per head row, known for D = 64 and 128, else -1. A
// thread's vectors are kThreads apart, so their (token, head) advance by a fixed step: no
// division per vector.
template <int kKind, bool kWrite, int kShift>
__global__ void __launch_bounds__(kThreads)
quant_kernel(const __grid_constant__ QuantArgs A, const __grid_constant__ ChunkList list) {
  constexpr int kPer = kWrite ? 16 : 8;      // elements per lane
  constexpr int kUnroll = kWrite ? 2 : 4;    // vectors in flight per thread
  pdl_wait();
  __shared__ int s_row[kQuantTokens];
  const int t0 = blockIdx.x * A.per_cta;
  const int nt = min(A.per_cta, list.row[list.n] - t0);
  if (static_cast<int>(threadIdx.x) < nt)
    s_row[threadIdx.x] = token_row(list, A.cache.pool, t0 + threadIdx.x, A.err);
  __syncthreads();
  pdl_trigger();
  const int li = blockIdx.y >> 1, kv = blockIdx.y & 1;
  constexpr bool kKnown = kShift > 0;
  const int shift = kKnown ? kShift : A.lane_shift;
  const int lanes = 1 << shift;
  const int H = A.g.H, D = kKnown ? kPer << kShift : A.g.D, E = A.g.E;
  // this layer's K or V in the pages; this CTA's first dense row
  const int64_t plane = (static_cast<int64_t>(A.layer_begin + li) * 2 + kv) *
                        A.cache.pool.num_pages * A.cache.pool.P;
  uint8_t* codes = reinterpret_cast<uint8_t*>(A.cache.pool.base) + plane * E;
  float* scale = A.cache.scale + plane * H;
  uint16_t* dense = (kv ? A.v : A.k) + (static_cast<int64_t>(li) * A.tokens + A.tok0 + t0) * E;
  const int rows = nt * H;                       // head rows of the CTA
  const int e0 = (threadIdx.x & (lanes - 1)) * kPer;  // elements of the thread's vectors
  const bool in_row = kKnown || e0 < D;
  int r = threadIdx.x >> shift;                  // the head row, its token and head
  int tok = static_cast<int>((static_cast<uint32_t>(r) * A.head_mul) >> 20);
  int h = r - tok * H;
  const int step = kThreads >> shift;
  const int step_tok = static_cast<int>((static_cast<uint32_t>(step) * A.head_mul) >> 20);
  const int step_h = step - step_tok * H;
  for (; r - (static_cast<int>(threadIdx.x) >> shift) < rows; ) {
    int row[kUnroll], hd[kUnroll], rr[kUnroll];  // page row (-1: unmapped, -2: nothing), head
    uint4 x[kUnroll][2];
    uint2 cw[kUnroll];
    float sc[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      row[u] = r < rows && in_row ? s_row[tok] : -2;
      hd[u] = h;
      rr[u] = r;
      x[u][0] = x[u][1] = make_uint4(0u, 0u, 0u, 0u);
      cw[u] = make_uint2(0u, 0u);
      sc[u] = 0.0f;
      if constexpr (kWrite) {
        if (row[u] > -2) {
          x[u][0] = ldg16(dense + r * D + e0);
          x[u][1] = ldg16(dense + r * D + e0 + 8);
        }
      } else if (row[u] >= 0) {
        cw[u] = __ldg(reinterpret_cast<const uint2*>(codes + static_cast<int64_t>(row[u]) * E +
                                                     (h * D + e0)));
        sc[u] = __ldg(scale + static_cast<int64_t>(row[u]) * H + h);
      }
      r += step;
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
        uint32_t m = __vmaxu2(magnitude8(x[u][0]), magnitude8(x[u][1]));
        if constexpr (kKnown) {
#pragma unroll
          for (int o = 1 << (kShift - 1); o > 0; o >>= 1)
            m = __vmaxu2(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
        } else {
          for (int o = lanes >> 1; o > 0; o >>= 1)
            m = __vmaxu2(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
        }
        const uint32_t top = max(m & 0xFFFFu, m >> 16);
        if (row[u] >= 0) {
          float s = row_scale<kKind>(top);
          uint4 c = make_uint4(0u, 0u, 0u, 0u);
          if (top < 0x7F80u) {
            float f[8];
            unpack8(x[u][0], f);
            const uint2 a = codes8<kKind>(f, s);
            unpack8(x[u][1], f);
            const uint2 b = codes8<kKind>(f, s);
            c = make_uint4(a.x, a.y, b.x, b.y);
          } else {             // a NaN or an infinity: the row reads back as NaN
            s = __uint_as_float(0x7FC00000u);
            if (e0 == 0) atomicOr(A.err, err_bit(TD_ERR_NONFINITE));
          }
          *reinterpret_cast<uint4*>(codes + static_cast<int64_t>(row[u]) * E + (hd[u] * D + e0)) = c;
          if (e0 == 0) scale[static_cast<int64_t>(row[u]) * H + hd[u]] = s;
        }
      } else {
        if (row[u] == -2) continue;
        // (an unmapped row: codes 0 and the scale 0, zeros)
        float y[8];
        values4<kKind>(cw[u].x, y);
        values4<kKind>(cw[u].y, y + 4);
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] = __fmul_rn(y[j], sc[u]);
        st16(dense + rr[u] * D + e0, pack8(y));
      }
    }
  }
}

template <int kKind, bool kWrite>
static cudaError_t run_kind(const QuantArgs& a, const ChunkList& list, dim3 grid,
                            cudaStream_t st) {
  constexpr int k64 = kWrite ? 2 : 3;
  if (a.g.D == 128)
    return launch_after(quant_kernel<kKind, kWrite, k64 + 1>, grid, kThreads, 0, st, a, list);
  if (a.g.D == 64)
    return launch_after(quant_kernel<kKind, kWrite, k64>, grid, kThreads, 0, st, a, list);
  return launch_after(quant_kernel<kKind, kWrite, -1>, grid, kThreads, 0, st, a, list);
}

template <bool kWrite>
static cudaError_t run(const QuantArgs& a, const ChunkList& list, CacheKind kind,
                       cudaStream_t st) {
  const int tokens = list.row[list.n];
  if (tokens == 0) return cudaSuccess;
  const dim3 grid((tokens + a.per_cta - 1) / a.per_cta, a.nl * 2);
  if (kind == kCacheInt8) return run_kind<kCacheInt8, kWrite>(a, list, grid, st);
  return run_kind<kCacheE4m3, kWrite>(a, list, grid, st);
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
