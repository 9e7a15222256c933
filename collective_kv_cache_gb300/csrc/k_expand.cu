// k_expand.cu - 8-bit pages unfolded for the tensor-core chunk attention: the KV tiles that a
// sequence's chunk sees, as dense bf16 tiles with a float scale per position and kv head.
//
// A long chunk is many tiles of query rows, and each would convert the same codes again. Here
// they are converted once: the codes are exact in bf16, so nothing is rounded. A position's
// scale stays a float of its own (it goes on the score or the weight), except where code *
// scale is exact in bf16 too: e4m3 with a power of two, as td_quantise_append writes it, is
// stored multiplied, with the scale 1. Positions that no token of the chunk sees become zeros
// with the scale 1, so that 0 * V is 0; a position of an unmapped page zeros with kHole.
//
// It reads a byte and writes two an element, once: bound by memory (four chunks' 26,000
// positions of 8 heads, D = 128: some 30 us of a 261 us call, 24 at a copy's rate). A CTA takes
// 16 positions of one layer's K or V, all heads (32: 264 us, 64: 268); a thread's vectors of 16
// codes are kThreads apart, four in flight (two as fast, eight 266).
#include "td_cache8.cuh"

namespace td {

namespace {

constexpr int kThreads = 256;
constexpr int kPositions = 16;

}  // namespace

template <int D, int kKind>
__global__ void __launch_bounds__(kThreads)
expand_kernel(const __grid_constant__ ChunkArgs A, const __grid_constant__ ChunkList list,
              const __grid_constant__ DenseTiles dense) {
  constexpr int kVec = D / 16;                      // vectors per head row
  constexpr int kStep = kThreads / kVec;            // head rows between a thread's vectors
  constexpr int kUnroll = 4;
  __shared__ int s_row[kPositions];
  pdl_wait();
  const int tid = threadIdx.x;
  constexpr int kPer = 128 / kPositions;
  const int tile = blockIdx.x / kPer, first = (blockIdx.x % kPer) * kPositions;
  const int li = blockIdx.y >> 1, kv = blockIdx.y & 1;
  const PoolDev& P = A.pool;
  if (tid < kPositions) {
    int x = 0;
    for (int hi = list.n - 1; x < hi;) {
      const int mid = (x + hi + 1) >> 1;
      if (dense.base[mid] <= tile) x = mid;
      else hi = mid - 1;
    }
    const int start = list.start[x], len = list.row[x + 1] - list.row[x];
    const DenseSpan span = dense_span(start, len, A.window, A.n_sink);
    const int pos = span.tile(tile - dense.base[x]) * 128 + first + tid;
    int row = -1;
    if (pos < start + len && (A.window == 0 || pos > start - A.window || pos < A.n_sink)) {
      const int lp = P.p_shift >= 0 ? (pos >> P.p_shift) : pos / P.P;
      const int page = lp < P.max_lp
                           ? __ldg(P.bt + static_cast<int64_t>(list.agent[x]) * P.max_lp + lp)
                           : -1;
      if (page < 0 || page >= P.num_pages) {
        atomicOr(A.err, err_bit(TD_ERR_UNMAPPED_PAGE));
        row = -2;
      } else {
        row = page * P.P + (pos - lp * P.P);
      }
    }
    s_row[tid] = row;
  }
  __syncthreads();
  pdl_trigger();
  const int H = A.g.H, E = A.g.E;
  const int64_t plane = (static_cast<int64_t>(A.layer_begin + li) * 2 + kv) * P.num_pages * P.P;
  const uint8_t* codes = reinterpret_cast<const uint8_t*>(P.base) + plane * E;
  const float* scale = A.scale + plane * H;
  const int64_t out_plane = static_cast<int64_t>(li) * 2 + kv;
  const int out_first = tile * 128 + first;
  uint16_t* out = A.dense + (out_plane * A.dense_rows + out_first) * E;
  // a scale that goes into the values: the products are exact, and no subnormal
  auto folds = [](float s) {
    return kKind == kCacheE4m3 && (__float_as_uint(s) & 0x007FFFFFu) == 0 && s >= 0x1p-100f &&
           s <= 128.0f;
  };
  // the scales, positions side by side
  for (int i = tid; i < kPositions * H; i += kThreads) {
    const int r = i % kPositions, h = i / kPositions, row = s_row[r];
    uint32_t bits = row == -2 ? kHole : 0x3F800000u;
    if (row >= 0) {
      const float s = __ldg(scale + static_cast<int64_t>(row) * H + h);
      // (a NaN is made the usual one, which is not kHole)
      if (!folds(s)) bits = s != s ? 0x7FFFFFFFu : __float_as_uint(s);
    }
    A.dense_scale[(out_plane * H + h) * A.dense_rows + out_first + r] = __uint_as_float(bits);
  }
  const int c = (tid % kVec) * 16;
  int n = tid / kVec;                               // the head row within the CTA's
  int r = n / H, h = n - r * H;
  const int step_r = kStep / H, step_h = kStep - step_r * H;
  const int rows = kPositions * H;
  for (; n < rows;) {
    int at[kUnroll], to[kUnroll];
    uint4 q[kUnroll];
    float s[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      at[u] = n < rows ? s_row[r] : -3;
      to[u] = n * D + c;
      q[u] = make_uint4(0u, 0u, 0u, 0u);
      s[u] = 1.0f;
      if (at[u] >= 0) {
        q[u] = __ldg(reinterpret_cast<const uint4*>(codes + static_cast<int64_t>(at[u]) * E +
                                                    (h * D + c)));
        if constexpr (kKind == kCacheE4m3) s[u] = __ldg(scale + static_cast<int64_t>(at[u]) * H + h);
      }
      n += kStep;
      r += step_r;
      h += step_h;
      if (h >= H) {
        h -= H;
        ++r;
      }
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      if (at[u] == -3) continue;
      uint4 a = make_uint4(0u, 0u, 0u, 0u), b = a;
      if (at[u] >= 0) {
        uint32_t f = kE4m3Factor;
        if constexpr (kKind == kCacheE4m3) {
          const uint32_t g = __float_as_uint(s[u] * 0x1p120f) >> 16;
          if (folds(s[u])) f = g | (g << 16);
        }
        a = make_uint4(word_bf16<kKind, false>(q[u].x, f), word_bf16<kKind, true>(q[u].x, f),
                       word_bf16<kKind, false>(q[u].y, f), word_bf16<kKind, true>(q[u].y, f));
        b = make_uint4(word_bf16<kKind, false>(q[u].z, f), word_bf16<kKind, true>(q[u].z, f),
                       word_bf16<kKind, false>(q[u].w, f), word_bf16<kKind, true>(q[u].w, f));
      }
      st16(out + to[u], a);
      st16(out + to[u] + 8, b);
    }
  }
}

cudaError_t launch_expand(const ChunkArgs& a, const ChunkList& list, const DenseTiles& dense,
                          CacheKind kind, cudaStream_t st) {
  const dim3 grid(static_cast<unsigned>(dense.base[list.n]) * (128 / kPositions), a.nl * 2);
  const bool wide = a.g.D == 128;
  if (kind == kCacheInt8)
    return wide ? launch_after(expand_kernel<128, kCacheInt8>, grid, kThreads, 0, st, a, list, dense)
                : launch_after(expand_kernel<64, kCacheInt8>, grid, kThreads, 0, st, a, list, dense);
  return wide ? launch_after(expand_kernel<128, kCacheE4m3>, grid, kThreads, 0, st, a, list, dense)
              : launch_after(expand_kernel<64, kCacheE4m3>, grid, kThreads, 0, st, a, list, dense);
}

}  // namespace td
