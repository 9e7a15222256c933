// k_chunk.cu - attention of a chunk of new tokens over a paged cache: the streaming kernel for
// a few query rows, and the join of its parts.
//
// Token u of a sequence's chunk sits at position pos = start + u and sees the positions
// p <= pos; under a window W only p > pos - W and the first n_sink positions. With
// s_p = scale q . k_p over the visible p: out = sum_p softmax(s)_p v_p, lse = ln sum_p e^{s_p}.
// 8-bit pages hold k = ks_p * code and v = vs_p * code: the codes are exact in bf16, so they
// go through the same products, with ks_p on the score and vs_p on the weight.
//
// One warp takes a unit = (layer, kv head, tile of 8 or 16 query rows, `span` of the tile's
// visible positions), 16 positions a step; the rows of a tile are (token, head of the group)
// pairs, so the group's heads share every read. It is bound by the pages' bytes, so nothing is
// staged: each lane loads 16-byte vectors of K and V straight into the registers of its
// fragments (mma.sync m16n8k16, positions or dims as the 16 rows, query rows as the 8
// columns). That works because a dot product may take its dims in any order: the lane's
// vector of 8 (or 16) neighbouring dims is read as the scattered dims of its fragment, the
// query's fragments and the output's rows are permuted alike, and V's pairs of positions
// are made with byte permutes. The next step's K is loaded once the scores have consumed
// this one's, its V after the weighted sum, so a warp has 8 KB under way at all times.
// The scores of a column are over the warp's positions, so the running maximum takes three
// shuffles and the weights turn into the next product's operand by two movmatrix. The
// weights are split in two bf16 parts (16 bits kept), two products, which costs nothing here.
//
// A position that no row of the tile sees is not read: its page may be unmapped and its bytes
// anything. A V row that some rows of the tile see and others do not may hold infinities or
// NaNs of its own; they must not reach the others through 0 * NaN, so in steps that mask
// anything such values leave the product and are added to the rows that see them alone.
#include "td_cache8.cuh"

namespace td {

namespace {

constexpr int kWarps = 4;
constexpr int kStep = 16;    // positions per step

__device__ __forceinline__ void mma_bf16(float* d, uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, "
      "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// An 8 x 8 matrix of 16-bit values over the warp (lane 4 r + c holds row r, columns 2c, 2c + 1)
// transposed.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

__device__ __forceinline__ bool nonfinite2(uint32_t w) {
  return (w & 0x7F80u) == 0x7F80u || (w & 0x7F800000u) == 0x7F800000u;
}

// What a lane holds of one kind of page.
template <int D, int kKind>
struct Layout {
  static constexpr bool k8 = kKind != kCacheBf16;
  // K: 16-byte vectors per row and lane, words (dim pairs) per vector
  static constexpr int kChunks = k8 ? D / 64 : D / 32;
  // V: neighbouring dims per vector and vectors per row and lane
  static constexpr int vDims = k8 ? D / 8 : 8;
  static constexpr int vChunks = D / (8 * vDims);
  static constexpr int vWords = k8 ? vDims / 4 : vDims / 2;
};

}  // namespace

template <int D, int kKind, int NB>
__global__ void __launch_bounds__(kWarps * 32)
chunk_rows_kernel(const __grid_constant__ ChunkArgs A, const __grid_constant__ ChunkList list,
                  const __grid_constant__ ChunkUnits units) {
  pdl_wait();
  using Y = Layout<D, kKind>;
  constexpr int KCH = D / 16;
  constexpr int R = 8 * NB;
  const int lane = threadIdx.x & 31;
  const int gid = lane >> 2, tig = lane & 3;
  const int total = units.base[list.n];
  const int64_t unit = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  if (unit >= static_cast<int64_t>(A.nl) * A.g.H * total) return;
  const int c = static_cast<int>(unit % total);
  const int64_t lh = unit / total;
  const int h = static_cast<int>(lh % A.g.H), li = static_cast<int>(lh / A.g.H);
  int x = 0;
  for (int hi = list.n - 1; x < hi;) {
    const int mid = (x + hi + 1) >> 1;
    if (units.base[mid] <= c) x = mid;
    else hi = mid - 1;
  }
  const int ns = units.nsplit[x];
  const int tile = (c - units.base[x]) / ns;
  const int split = c - units.base[x] - tile * ns;
  const int len = list.row[x + 1] - list.row[x], start = list.start[x];
  const int rows = len * A.G;
  const int r0 = tile * R;

  // the tile's visible positions, numbered v: the first `sinks`, then lo .. p_last
  const int p_first = start + r0 / A.G;
  const int p_last = start + min(r0 + R - 1, rows - 1) / A.G;
  const int lo = A.window ? max(0, p_first - A.window + 1) : 0;
  const int sinks = A.window ? min(A.n_sink, lo) : 0;
  const int n_vis = sinks + p_last + 1 - lo;
  const int v0 = split * A.span;
  const int v1 = min(v0 + A.span, n_vis);

  // this lane's query rows: as a B-operand column (gid), and as accumulator columns
  int pos_q[NB][2];          // positions of columns 2 tig, 2 tig + 1; -1 past the last row
  uint32_t qf[NB][KCH][2];
#pragma unroll
  for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int r = r0 + nb * 8 + 2 * tig + e;
      pos_q[nb][e] = r < rows ? start + r / A.G : -1;
    }
    const int r = r0 + nb * 8 + gid;
    const bool live = r < rows;
    const int tok = live ? r / A.G : 0;
    const int64_t row = static_cast<int64_t>(li) * A.tokens + list.tok[x] + tok;
    const uint16_t* q = A.q + (row * A.nq + h * A.G + (live ? r - tok * A.G : 0)) * D;
#pragma unroll
    for (int kc = 0; kc < KCH; ++kc)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        // the dims that the lane's K vector gives to fragment kc, register pair e
        const int dim = Y::k8 ? ((kc >> 2) * 4 + tig) * 16 + (kc & 3) * 4 + e * 2
                              : ((kc >> 1) * 4 + tig) * 8 + (kc & 1) * 4 + e * 2;
        qf[nb][kc][e] = live ? __ldg(reinterpret_cast<const unsigned int*>(q + dim)) : 0u;
      }
  }

  const PoolDev& P = A.pool;
  const int64_t plane = (static_cast<int64_t>(A.layer_begin + li) * 2) * P.num_pages * P.P;
  const int64_t vplane = plane + P.num_pages * P.P;
  const int E = A.g.E;
  // bytes of an element: 2 or 1
  const uint8_t* kbase = reinterpret_cast<const uint8_t*>(P.base) +
                         (plane * E + h * D) * (Y::k8 ? 1 : 2);
  const uint8_t* vbase = reinterpret_cast<const uint8_t*>(P.base) +
                         (vplane * E + h * D) * (Y::k8 ? 1 : 2);
  const float* kscale = Y::k8 ? A.scale + plane * A.g.H + h : nullptr;
  const float* vscale = Y::k8 ? A.scale + vplane * A.g.H + h : nullptr;
  const int row_bytes = E * (Y::k8 ? 1 : 2);

  // position of index v, and lane l < 16's page row of index v + l (-1: not visible, unmapped)
  auto position = [&](int v) { return v < sinks ? v : lo + v - sinks; };
  auto page_row = [&](int v) {
    const int vi = v + (lane & 15);
    if (vi >= v1) return -1;
    const int pos = position(vi);
    const int lp = P.p_shift >= 0 ? (pos >> P.p_shift) : pos / P.P;
    int32_t page = -1;
    if (lp < P.max_lp) page = __ldg(P.bt + static_cast<int64_t>(list.agent[x]) * P.max_lp + lp);
    if (page < 0 || page >= P.num_pages) {
      atomicOr(A.err, err_bit(TD_ERR_UNMAPPED_PAGE));
      return -1;
    }
    return page * P.P + (pos - lp * P.P);
  };

  uint4 kr[2][Y::kChunks];                 // rows gid, gid + 8
  uint32_t vr[4][Y::vChunks][Y::vWords];   // rows 2 tig, 2 tig + 1, 2 tig + 8, 2 tig + 9
  float ks[2] = {1.0f, 1.0f}, vs[2] = {1.0f, 1.0f};   // scales of rows gid, gid + 8
  auto load_k = [&](int rows_of) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int row = __shfl_sync(0xFFFFFFFFu, rows_of, gid + 8 * i);
      const uint8_t* p = kbase + static_cast<int64_t>(row) * row_bytes;
#pragma unroll
      for (int j = 0; j < Y::kChunks; ++j)
        kr[i][j] = row < 0 ? make_uint4(0u, 0u, 0u, 0u)
                           : __ldg(reinterpret_cast<const uint4*>(p) + j * 4 + tig);
      if constexpr (Y::k8) {
        ks[i] = row < 0 ? 0.0f : __ldg(kscale + static_cast<int64_t>(row) * A.g.H);
        vs[i] = row < 0 ? 0.0f : __ldg(vscale + static_cast<int64_t>(row) * A.g.H);
      }
    }
  };
  auto load_v = [&](int rows_of) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int row = __shfl_sync(0xFFFFFFFFu, rows_of, 2 * tig + (i & 1) + 8 * (i >> 1));
      const uint8_t* p = vbase + static_cast<int64_t>(row) * row_bytes;
#pragma unroll
      for (int j = 0; j < Y::vChunks; ++j) {
        if constexpr (Y::vWords == 4) {
          const uint4 w = row < 0 ? make_uint4(0u, 0u, 0u, 0u)
                                  : __ldg(reinterpret_cast<const uint4*>(p) + j * 8 + gid);
          vr[i][j][0] = w.x;
          vr[i][j][1] = w.y;
          vr[i][j][2] = w.z;
          vr[i][j][3] = w.w;
        } else {
          const uint2 w = row < 0 ? make_uint2(0u, 0u)
                                  : __ldg(reinterpret_cast<const uint2*>(p) + j * 8 + gid);
          vr[i][j][0] = w.x;
          vr[i][j][1] = w.y;
        }
      }
    }
  };

  // O^T: acc[nb][mt] = dims (lane's dims 2 mt, 2 mt + 1) x rows 2 tig, 2 tig + 1
  float acc[NB][KCH][4];
  float m_run[NB][2], l_part[NB][2];
#pragma unroll
  for (int nb = 0; nb < NB; ++nb) {
    m_run[nb][0] = m_run[nb][1] = -INFINITY;
    l_part[nb][0] = l_part[nb][1] = 0.0f;
#pragma unroll
    for (int mt = 0; mt < KCH; ++mt)
      acc[nb][mt][0] = acc[nb][mt][1] = acc[nb][mt][2] = acc[nb][mt][3] = 0.0f;
  }

  int cur = page_row(v0), nxt = page_row(v0 + kStep);
  if (v0 < v1) {
    load_k(cur);
    load_v(cur);
  }
  for (int v = v0; v < v1; v += kStep) {
    // scores of positions gid, gid + 8 against rows 2 tig, 2 tig + 1
    float s[NB][4];
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) s[nb][0] = s[nb][1] = s[nb][2] = s[nb][3] = 0.0f;
#pragma unroll
    for (int kc = 0; kc < KCH; ++kc) {
      uint32_t a[4];
      if constexpr (Y::k8) {
        const int j = kc >> 2;
        const uint32_t w0 = reinterpret_cast<const uint32_t*>(&kr[0][j])[kc & 3];
        const uint32_t w1 = reinterpret_cast<const uint32_t*>(&kr[1][j])[kc & 3];
        a[0] = word_bf16<kKind, false>(w0);
        a[1] = word_bf16<kKind, false>(w1);
        a[2] = word_bf16<kKind, true>(w0);
        a[3] = word_bf16<kKind, true>(w1);
      } else {
        const uint32_t* w0 = reinterpret_cast<const uint32_t*>(&kr[0][kc >> 1]) + (kc & 1) * 2;
        const uint32_t* w1 = reinterpret_cast<const uint32_t*>(&kr[1][kc >> 1]) + (kc & 1) * 2;
        a[0] = w0[0];
        a[1] = w1[0];
        a[2] = w0[1];
        a[3] = w1[1];
      }
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
        mma_bf16(s[nb], a[0], a[1], a[2], a[3], qf[nb][kc][0], qf[nb][kc][1]);
    }
    const float kse[2] = {ks[0], ks[1]}, vse[2] = {vs[0], vs[1]};
    const int mapped[2] = {__shfl_sync(0xFFFFFFFFu, cur, gid),
                           __shfl_sync(0xFFFFFFFFu, cur, gid + 8)};
    const int nn = page_row(v + 2 * kStep);
    if (v + kStep < v1) load_k(nxt);
    // the weights: masked, in base 2 under the running maximum
    const int pos[2] = {position(v + gid), position(v + gid + 8)};
    bool masks = false;
    float p[NB][4], fac[NB][2];
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int pq = pos_q[nb][i & 1], pp = pos[i >> 1];
        const bool ok = mapped[i >> 1] >= 0 && pp <= pq &&
                        (A.window == 0 || pp > pq - A.window || pp < A.n_sink);
        masks |= !ok && pq >= 0;
        const float k = Y::k8 ? __fmul_rn(s[nb][i], kse[i >> 1]) : s[nb][i];
        s[nb][i] = ok ? __fmul_rn(k, A.scale_log2) : -INFINITY;
        p[nb][i] = ok ? 1.0f : 0.0f;
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float mx = fmaxf(s[nb][e], s[nb][e + 2]);
        mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 4));
        mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 8));
        mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 16));
        const float m_new = fmaxf(m_run[nb][e], mx);
        fac[nb][e] = m_run[nb][e] == -INFINITY ? 0.0f : exp2f(m_run[nb][e] - m_new);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float w = s[nb][e + 2 * i] == -INFINITY ? 0.0f : exp2f(s[nb][e + 2 * i] - m_new);
          s[nb][e + 2 * i] = w;
        }
        l_part[nb][e] = __fmaf_rn(l_part[nb][e], fac[nb][e], s[nb][e] + s[nb][e + 2]);
        m_run[nb][e] = m_new;
      }
      // the weight on V: with the row's scale, 0 where the row is not seen
#pragma unroll
      for (int i = 0; i < 4; ++i)
        p[nb][i] = p[nb][i] == 0.0f ? 0.0f : (Y::k8 ? __fmul_rn(s[nb][i], vse[i >> 1]) : s[nb][i]);
    }
    uint32_t ph[NB][2], pl[NB][2];
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint32_t hi = pack_bf2(p[nb][2 * i], p[nb][2 * i + 1]);
        const uint32_t lo2 = pack_bf2(__fsub_rn(p[nb][2 * i], bf_lo(hi)),
                                      __fsub_rn(p[nb][2 * i + 1], bf_hi(hi)));
        ph[nb][i] = transpose8(hi);
        pl[nb][i] = transpose8(lo2);
      }
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int mt = 0; mt < KCH; ++mt) {
        acc[nb][mt][0] *= fac[nb][0];
        acc[nb][mt][1] *= fac[nb][1];
        acc[nb][mt][2] *= fac[nb][0];
        acc[nb][mt][3] *= fac[nb][1];
      }
    if constexpr (!Y::k8) {
      // values that must not meet a zero weight (rare: a step that masks, with such a value)
      if (__any_sync(0xFFFFFFFFu, masks)) {
        bool bad = false;
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < Y::vChunks; ++j)
#pragma unroll
            for (int w = 0; w < Y::vWords; ++w) bad |= nonfinite2(vr[i][j][w]);
        if (__any_sync(0xFFFFFFFFu, bad)) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            for (int t = 0; t < 4; ++t) {
              // position k of the step: its V is held by the quad's lane t
              const int k = 2 * t + (i & 1) + 8 * (i >> 1);
              float pk[NB][2];
#pragma unroll
              for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                for (int e = 0; e < 2; ++e)
                  pk[nb][e] = __shfl_sync(0xFFFFFFFFu, p[nb][e + 2 * (i >> 1)], (k & 7) * 4 + tig);
#pragma unroll
              for (int j = 0; j < Y::vChunks; ++j)
#pragma unroll
                for (int w = 0; w < Y::vWords; ++w) {
                  const uint32_t vw = __shfl_sync(0xFFFFFFFFu, vr[i][j][w], (lane & ~3) | t);
                  const int mt = j * Y::vWords + w;
#pragma unroll
                  for (int half = 0; half < 2; ++half) {
                    const float val = half ? bf_hi(vw) : bf_lo(vw);
                    if ((__float_as_uint(val) & 0x7F800000u) != 0x7F800000u) continue;
#pragma unroll
                    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                      for (int e = 0; e < 2; ++e)
                        if (pk[nb][e] != 0.0f)
                          acc[nb][mt][half * 2 + e] = __fmaf_rn(pk[nb][e], val, acc[nb][mt][half * 2 + e]);
                  }
                }
            }
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < Y::vChunks; ++j)
#pragma unroll
              for (int w = 0; w < Y::vWords; ++w) {
                uint32_t z = vr[i][j][w];
                if ((z & 0x7F80u) == 0x7F80u) z &= 0xFFFF0000u;
                if ((z & 0x7F800000u) == 0x7F800000u) z &= 0x0000FFFFu;
                vr[i][j][w] = z;
              }
        }
      }
    }
#pragma unroll
    for (int mt = 0; mt < KCH; ++mt) {
      uint32_t a[4];
      if constexpr (Y::k8) {
        const int w = mt >> 1, i0 = (mt & 1) * 2;   // word and first byte of dims 2 mt, 2 mt + 1
        a[0] = pair_bf16<kKind>(vr[0][0][w], vr[1][0][w], i0);
        a[1] = pair_bf16<kKind>(vr[0][0][w], vr[1][0][w], i0 + 1);
        a[2] = pair_bf16<kKind>(vr[2][0][w], vr[3][0][w], i0);
        a[3] = pair_bf16<kKind>(vr[2][0][w], vr[3][0][w], i0 + 1);
      } else {
        const int j = mt / Y::vWords, w = mt % Y::vWords;
        a[0] = __byte_perm(vr[0][j][w], vr[1][j][w], 0x5410);
        a[1] = __byte_perm(vr[0][j][w], vr[1][j][w], 0x7632);
        a[2] = __byte_perm(vr[2][j][w], vr[3][j][w], 0x5410);
        a[3] = __byte_perm(vr[2][j][w], vr[3][j][w], 0x7632);
      }
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        mma_bf16(acc[nb][mt], a[0], a[1], a[2], a[3], ph[nb][0], ph[nb][1]);
        mma_bf16(acc[nb][mt], a[0], a[1], a[2], a[3], pl[nb][0], pl[nb][1]);
      }
    }
    if (v + kStep < v1) load_v(nxt);
    cur = nxt;
    nxt = nn;
  }

  // the lane's dims: vector j holds dims (j * 8 + gid) * vDims + 0 .. vDims - 1
#pragma unroll
  for (int nb = 0; nb < NB; ++nb)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float l = l_part[nb][e];
      l += __shfl_xor_sync(0xFFFFFFFFu, l, 4);
      l += __shfl_xor_sync(0xFFFFFFFFu, l, 8);
      l += __shfl_xor_sync(0xFFFFFFFFu, l, 16);
      const int rt = nb * 8 + 2 * tig + e;
      const int r = r0 + rt;
      if (r >= rows) continue;
      if (A.direct) {
        const int tok = r / A.G;
        const int64_t row =
            (static_cast<int64_t>(li) * A.tokens + list.tok[x] + tok) * A.nq + h * A.G +
            (r - tok * A.G);
        const float inv = l == 0.0f ? 0.0f : 1.0f / l;    // a row that sees nothing: zeros
#pragma unroll
        for (int j = 0; j < Y::vChunks; ++j)
#pragma unroll
          for (int w = 0; w < Y::vDims / 8; ++w) {
            uint32_t o[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int mt = j * (Y::vDims / 2) + w * 4 + i;
              o[i] = pack_bf2(acc[nb][mt][e] * inv, acc[nb][mt][2 + e] * inv);
            }
            st16(A.out + row * D + (j * 8 + gid) * Y::vDims + w * 8,
                 make_uint4(o[0], o[1], o[2], o[3]));
          }
        if (gid == 0 && A.lse)
          A.lse[row] = l == 0.0f ? -INFINITY : (m_run[nb][e] + log2f(l)) * 0.69314718055994530942f;
      } else {
        float* po = A.part_o + (unit * R + rt) * D;
#pragma unroll
        for (int j = 0; j < Y::vChunks; ++j)
#pragma unroll
          for (int w = 0; w < Y::vDims / 4; ++w) {
            const int mt = j * (Y::vDims / 2) + w * 2;
            *reinterpret_cast<float4*>(po + (j * 8 + gid) * Y::vDims + w * 4) =
                make_float4(acc[nb][mt][e], acc[nb][mt][2 + e], acc[nb][mt + 1][e],
                            acc[nb][mt + 1][2 + e]);
          }
        if (gid == 0) {
          A.part_ml[(unit * R + rt) * 2] = m_run[nb][e];
          A.part_ml[(unit * R + rt) * 2 + 1] = l;
        }
      }
    }
}

// One warp per (layer, token, query head): the row's parts joined. A part that saw nothing has
// the maximum -inf and weight 0, and is not read.
template <int D>
__global__ void __launch_bounds__(128)
chunk_join_kernel(const __grid_constant__ ChunkArgs A, const __grid_constant__ ChunkList list,
                  const __grid_constant__ ChunkUnits units, int R) {
  pdl_wait();
  constexpr int DPL = D / 32;
  const int lane = threadIdx.x & 31;
  const int n_tok = list.row[list.n];
  const int64_t w = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 5);
  if (w >= static_cast<int64_t>(A.nl) * n_tok * A.nq) return;
  const int gq = static_cast<int>(w % A.nq);
  const int t = static_cast<int>((w / A.nq) % n_tok);
  const int li = static_cast<int>(w / (static_cast<int64_t>(A.nq) * n_tok));
  int x = 0;
  for (int hi = list.n - 1; x < hi;) {
    const int mid = (x + hi + 1) >> 1;
    if (list.row[mid] <= t) x = mid;
    else hi = mid - 1;
  }
  const int h = gq / A.G;
  const int r = (t - list.row[x]) * A.G + gq - h * A.G;
  const int tile = r / R, rt = r - tile * R;
  const int ns = units.nsplit[x];
  const int64_t u0 = (static_cast<int64_t>(li) * A.g.H + h) * units.base[list.n] + units.base[x] +
                     static_cast<int64_t>(tile) * ns;
  float mx = -INFINITY;
  bool nan = false;
  for (int i = lane; i < ns; i += 32) {
    const float m = A.part_ml[((u0 + i) * R + rt) * 2];
    mx = fmaxf(mx, m);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, o));
  float l = 0.0f, acc[DPL];
#pragma unroll
  for (int d = 0; d < DPL; ++d) acc[d] = 0.0f;
  for (int i0 = 0; i0 < ns; i0 += 32) {
    float wgt = 0.0f;
    if (i0 + lane < ns) {
      const float* ml = A.part_ml + ((u0 + i0 + lane) * R + rt) * 2;
      // a part whose scores are NaN keeps the maximum -inf but a sum that is NaN
      nan |= ml[1] != ml[1];
      wgt = ml[0] == -INFINITY ? 0.0f : exp2f(ml[0] - mx);
      l = wgt == 0.0f ? l : __fmaf_rn(ml[1], wgt, l);
    }
    const int nb = min(32, ns - i0);
#pragma unroll 4
    for (int j = 0; j < nb; ++j) {
      const float wj = __shfl_sync(0xFFFFFFFFu, wgt, j);
      if (wj == 0.0f) continue;
      const float* po = A.part_o + ((u0 + i0 + j) * R + rt) * D + lane * DPL;
      if constexpr (DPL == 4) {
        const float4 q = *reinterpret_cast<const float4*>(po);
        acc[0] = __fmaf_rn(q.x, wj, acc[0]);
        acc[1] = __fmaf_rn(q.y, wj, acc[1]);
        acc[2] = __fmaf_rn(q.z, wj, acc[2]);
        acc[3] = __fmaf_rn(q.w, wj, acc[3]);
      } else {
        const float2 q = *reinterpret_cast<const float2*>(po);
        acc[0] = __fmaf_rn(q.x, wj, acc[0]);
        acc[1] = __fmaf_rn(q.y, wj, acc[1]);
      }
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xFFFFFFFFu, l, o);
  if (__any_sync(0xFFFFFFFFu, nan)) l = __uint_as_float(0x7FC00000u);
  const int64_t row =
      (static_cast<int64_t>(li) * A.tokens + list.tok[x] + t - list.row[x]) * A.nq + gq;
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
  uint32_t* out = reinterpret_cast<uint32_t*>(A.out + row * D + lane * DPL);
#pragma unroll
  for (int d = 0; d < DPL; d += 2) out[d / 2] = pack_bf2(acc[d] * inv, acc[d + 1] * inv);
  if (lane == 0 && A.lse)
    A.lse[row] = l == 0.0f ? -INFINITY : (mx + log2f(l)) * 0.69314718055994530942f;
}

template <int D, int kKind>
static cudaError_t run_rows(const ChunkArgs& a, const ChunkList& list, const ChunkUnits& units,
                            int rows_per_tile, cudaStream_t st) {
  const int64_t n = static_cast<int64_t>(a.nl) * a.g.H * units.base[list.n];
  if (n == 0) return cudaSuccess;
  const unsigned grid = static_cast<unsigned>((n + kWarps - 1) / kWarps);
  if (rows_per_tile == 8)
    return launch_after(chunk_rows_kernel<D, kKind, 1>, grid, kWarps * 32, 0, st, a, list, units);
  return launch_after(chunk_rows_kernel<D, kKind, 2>, grid, kWarps * 32, 0, st, a, list, units);
}

cudaError_t launch_chunk_rows(const ChunkArgs& a, const ChunkList& list, const ChunkUnits& units,
                              CacheKind kind, int rows_per_tile, cudaStream_t st) {
  if (a.g.D != 64 && a.g.D != 128) return cudaErrorInvalidValue;
  const bool wide = a.g.D == 128;
  switch (kind) {
    case kCacheBf16:
      return wide ? run_rows<128, kCacheBf16>(a, list, units, rows_per_tile, st)
                  : run_rows<64, kCacheBf16>(a, list, units, rows_per_tile, st);
    case kCacheInt8:
      return wide ? run_rows<128, kCacheInt8>(a, list, units, rows_per_tile, st)
                  : run_rows<64, kCacheInt8>(a, list, units, rows_per_tile, st);
    case kCacheE4m3:
      return wide ? run_rows<128, kCacheE4m3>(a, list, units, rows_per_tile, st)
                  : run_rows<64, kCacheE4m3>(a, list, units, rows_per_tile, st);
  }
  return cudaErrorInvalidValue;
}

cudaError_t launch_chunk_join(const ChunkArgs& a, const ChunkList& list, const ChunkUnits& units,
                              int rows_per_tile, cudaStream_t st) {
  const int64_t rows = static_cast<int64_t>(a.nl) * list.row[list.n] * a.nq;
  const unsigned grid = static_cast<unsigned>((rows + 3) / 4);
  if (a.g.D == 128)
    return launch_after(chunk_join_kernel<128>, grid, 128, 0, st, a, list, units, rows_per_tile);
  return launch_after(chunk_join_kernel<64>, grid, 128, 0, st, a, list, units, rows_per_tile);
}

}  // namespace td
