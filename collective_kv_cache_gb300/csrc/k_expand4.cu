// k_expand4.cu - 4-bit pages unfolded for the tensor-core chunk attention: the KV tiles that a
// sequence's chunk sees, as dense bf16 tiles with a float scale per position and kv head
// (k_expand.cu's layout).
//
// int4: code - zero, -15 to 15, is a bf16, and the row's scale stays a float of its own. e2m1: code *
// 2^(b - 127) is a bf16 as long as the row's four bytes are in [27, 227] (rows as
// td_quantise_slots writes them, up to 2^100), and is stored multiplied, with the scale 1; in other
// rows the quarters' powers of two relative to the largest go into the values and that one is the
// scale. Nothing is rounded either way, but a quarter 127 or more binades below its row's largest counts
// as 0. Positions that no token of the chunk sees become zeros with
// the scale 1, so that 0 * V is 0; a position of an unmapped page zeros with kHole.
//
// It reads 0.53 bytes and writes 2 an element, once: bound by memory. A CTA takes 32 positions of one
// layer's K or V, all heads; a lane two vectors of 8 elements, half a row apart (whole lines written), of
// two rows at a time. The 32 spans of 5 to 1505 rows on 244,000 positions of 8 heads at D = 128, in all,
// take 926 us over e2m1 pages; with 16 positions a CTA 934, with one vector a lane besides 951.
#include "td_cache4.cuh"

namespace td {

namespace {

constexpr int kThreads = 256;
constexpr int kPositions = 32;

}  // namespace

template <int D, int kKind>
__global__ void __launch_bounds__(kThreads)
expand4_kernel(const __grid_constant__ ChunkArgs A, const __grid_constant__ ChunkList list,
               const __grid_constant__ DenseTiles dense) {
  constexpr int kLanes = D / 16;                    // lanes per head row, two vectors of 8 each
  constexpr int kStep = kThreads / kLanes;          // head rows between a thread's
  constexpr int kUnroll = 2;
  __shared__ int2 s_at[kPositions];                 // page and slot; {-1, 0} unseen, {-2, 0} unmapped
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
    int2 at = make_int2(-1, 0);
    if (pos < start + len && (A.window == 0 || pos > start - A.window || pos < A.n_sink)) {
      const int lp = P.p_shift >= 0 ? (pos >> P.p_shift) : pos / P.P;
      const int page = lp < P.max_lp ? P.bt[static_cast<int64_t>(list.agent[x]) * P.max_lp + lp] : -1;
      if (page < 0 || page >= P.num_pages) {
        atomicOr(A.err, err_bit(TD_ERR_UNMAPPED_PAGE));
        at.x = -2;
      } else {
        at = make_int2(page, pos - lp * P.P);
      }
    }
    s_at[tid] = at;
  }
  __syncthreads();
  pdl_trigger();
  const int H = A.g.H, E = A.g.E;
  const int64_t plane = (static_cast<int64_t>(A.layer_begin + li) * 2 + kv) * P.num_pages * P.P * H;
  const uint8_t* codes = reinterpret_cast<const uint8_t*>(P.base) + plane * (D / 2);
  const uint32_t* words = A.word + plane;
  const int64_t out_plane = static_cast<int64_t>(li) * 2 + kv;
  const int out_first = tile * 128 + first;
  uint16_t* out = A.dense + (out_plane * A.dense_rows + out_first) * E;
  auto row_of = [&](const int2& at, int h) { return (at.x * H + h) * P.P + at.y; };
  // e2m1: every byte in [27, 227]
  auto folds = [](uint32_t w) {
    return __vminu4(w, 0x1B1B1B1Bu) == 0x1B1B1B1Bu && __vmaxu4(w, 0xE3E3E3E3u) == 0xE3E3E3E3u;
  };
  // the scales, positions side by side
  for (int i = tid; i < kPositions * H; i += kThreads) {
    const int r = i % kPositions, h = i / kPositions;
    const int2 at = s_at[r];
    uint32_t bits = at.x == -2 ? kHole : 0x3F800000u;
    if (at.x >= 0) {
      const uint32_t w = __ldg(words + row_of(at, h));
      float s = 1.0f;
      if constexpr (kKind == kCacheInt4) s = __uint_as_float(w & 0xFFFF0000u);
      else if (!folds(w)) s = byte_scale(largest_byte(w));
      // (a NaN is made the usual one, which is not kHole)
      bits = s != s ? 0x7FFFFFFFu : __float_as_uint(s);
    }
    A.dense_scale[(out_plane * H + h) * A.dense_rows + out_first + r] = __uint_as_float(bits);
  }
  const int part = tid % kLanes;
  int n = tid / kLanes;                             // the head row within the CTA's
  int r = n / H, h = n - r * H;
  const int step_r = kStep / H, step_h = kStep - step_r * H;
  const int rows = kPositions * H;
  while (n < rows) {
    int at[kUnroll], to[kUnroll];
    uint32_t q[kUnroll][2], w[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int2 place = n < rows ? s_at[r] : make_int2(-3, 0);
      at[u] = place.x < 0 ? place.x : row_of(place, h);
      to[u] = n * D + part * 8;
      q[u][0] = q[u][1] = w[u] = 0u;
      if (at[u] >= 0) {
        const uint32_t* from = reinterpret_cast<const uint32_t*>(codes + static_cast<int64_t>(at[u]) * (D / 2));
        q[u][0] = __ldg(from + part);
        q[u][1] = __ldg(from + part + kLanes);
        w[u] = __ldg(words + at[u]);
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
      const bool fold = folds(w[u]);
      const int big = static_cast<int>(largest_byte(w[u]));
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint32_t c = q[u][i];
        uint4 y = make_uint4(0u, 0u, 0u, 0u);
        if (at[u] >= 0) {
          if constexpr (kKind == kCacheInt4) {
            // 128 + code less 128 + zero: both have 8 bits
            const uint32_t z = 0x4300u | (w[u] & 0x7Fu), z2 = z | (z << 16);
            const uint32_t even = c & 0x0F0F0F0Fu, odd = (c >> 4) & 0x0F0F0F0Fu;
            auto two = [&](uint32_t pair) {
              uint32_t d;
              asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"((pair & 0x000F000Fu) | 0x43004300u), "r"(z2));
              return d;
            };
            y = make_uint4(two(__byte_perm(even, odd, 0x4400)), two(__byte_perm(even, odd, 0x5511)),
                           two(__byte_perm(even, odd, 0x6622)), two(__byte_perm(even, odd, 0x7733)));
          } else {
            const uint32_t b = (w[u] >> (8 * (part / (kLanes / 2) + 2 * i))) & 0xFFu;
            const uint32_t e = fold ? b : static_cast<uint32_t>(max(static_cast<int>(b) + 127 - big, 0));
            const float s = __uint_as_float(e << 23);
            auto two = [&](uint32_t h2) { return pack_bf2(f16_lo(h2) * s, f16_hi(h2) * s); };
            y = make_uint4(two(e2m1_f16<0>(c)), two(e2m1_f16<1>(c)), two(e2m1_f16<2>(c)),
                           two(e2m1_f16<3>(c)));
          }
        }
        st16(out + to[u] + i * kLanes * 8, y);
      }
    }
  }
}

cudaError_t launch_expand4(const ChunkArgs& a, const ChunkList& list, const DenseTiles& dense,
                           CacheKind kind, cudaStream_t st) {
  const dim3 grid(static_cast<unsigned>(dense.base[list.n]) * (128 / kPositions), a.nl * 2);
  const bool wide = a.g.D == 128;
  if (kind == kCacheInt4)
    return wide ? launch_after(expand4_kernel<128, kCacheInt4>, grid, kThreads, 0, st, a, list, dense)
                : launch_after(expand4_kernel<64, kCacheInt4>, grid, kThreads, 0, st, a, list, dense);
  return wide ? launch_after(expand4_kernel<128, kCacheE2m1>, grid, kThreads, 0, st, a, list, dense)
              : launch_after(expand4_kernel<64, kCacheE2m1>, grid, kThreads, 0, st, a, list, dense);
}

}  // namespace td
