// k_chunk.cu - attention of a chunk of new tokens over a paged cache: the streaming kernel for
// a few query rows, and the join of its parts.
//
// Token u of a sequence's chunk sits at position pos = start + u and sees the positions
// p <= pos; under a window W only p > pos - W and the first n_sink positions. With
// s_p = scale q . k_p over the visible p: out = sum_p softmax(s)_p v_p, lse = ln sum_p e^{s_p}.
// 8-bit pages hold k = ks_p * code and v = vs_p * code: the codes are exact in f16 and bf16, so
// they go through the same products (K in f16, V in bf16), with ks_p on the score and vs_p on
// the weight.
//
// A block takes a unit = (layer, kv head, tile of 8 or 16 query rows, `span` of the tile's
// visible positions), its four warps every fourth step of 16 or 32 positions each; they are
// joined in shared memory at the end, so that a unit leaves one partial result (a warp a unit
// left four times as many, whose join took 7.5 us of a 31 us call). The rows of a tile are
// (token, head of the group) pairs, so the group's heads share every read: the pages' bytes are
// its floor. Products are mma.sync m16n8k16, positions or dims as the 16 rows, query rows as
// the 8 columns; tcgen05's 128 rows would be idle for seven eighths or more. Each lane copies
// exactly the 16-byte vectors of K and V that its own fragments are made of (cp.async, rows out
// of sight zero-filled) into a ring of its own, and reads them back without any barrier. That
// works because a dot product may take its dims in any order: the lane's vector
// of 8 (or 16) neighbouring dims is read as the scattered dims of its fragment, the query's
// fragments and the output's rows are permuted alike, and V's pairs of positions are made with
// byte permutes. The ring keeps the next steps' copies under way during a step, and the block
// table is read a step ahead of the copies (loads straight into registers, with the table read
// in line, left a warp waiting some 6,000 cycles a step).
// The scores of a column are over the warp's positions, so the running maximum takes three
// shuffles and the weights turn into the next product's operand by two movmatrix. The
// weights are split in two bf16 parts (16 bits kept), two products, which costs nothing here.
//
// Measured on one GB300, 28 query heads on 4, D = 128: single tokens of 10 agents after 3060 to
// 6560 positions take 26 us (3.7 TB/s, half the copy rate: a few steps a warp, so the latency
// of the table, the pages and the join are most of it; td_paged_attention's kernel takes 38 us
// over the same pages). Over int8 pages, 64 agents after 8192 to 24576 positions, 230 us
// (4.7 TB/s, 70% of the copy rate). No unit is full there (ALU 56%, issue 54% of the cycles);
// of the 4.8 cycles between a warp's issues only 0.4 wait for the pages, the others for results
// (0.9), shared memory (0.6), a busy pipe (0.7) or another warp (0.8): it is the arithmetic,
// the codes' conversion most of it, of three warps a scheduler.
//
// A position that no row of the tile sees is not read: its page may be unmapped and its bytes
// anything. A V row that some rows of the tile see and others do not may hold infinities or
// NaNs of its own; they must not reach the others through 0 * NaN, so in steps that mask
// anything such values leave the product and are added to the rows that see them alone.
#include "td_cache8.cuh"

namespace td {

namespace {

__device__ __forceinline__ void mma_bf16(float* d, uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, "
      "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void mma_f16(float* d, uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, "
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

// 16 (4) bytes into shared memory, or zeros where `live` is not set.
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool live) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(live ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void copy4(uint32_t dst, const void* src, bool live) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src),
               "r"(live ? 4 : 0)
               : "memory");
}

// Four 8 x 8 matrices of 16-bit values, transposed: lane l names row l & 7 of matrix l >> 3.
__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t* r, uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// The larger one, a NaN if either is.
__device__ __forceinline__ float max_nan(float a, float b) {
  float y;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
  return y;
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
  static constexpr int vBytes = vWords * 4;
  // a step takes `subs` times 16 positions; its bytes in shared memory: per sub-step and lane
  // 2 rows of K and 4 of V, then the positions' scales
  static constexpr int subs = !k8 && D == 128 ? 1 : 2;
  static constexpr int step = 16 * subs;
  static constexpr int kBytes = 2 * kChunks * 16 * 32;
  static constexpr int vAll = 4 * vChunks * vBytes * 32;
  static constexpr int codes = subs * (kBytes + vAll);
  static constexpr int stage = codes + (k8 ? 2 * step * 4 : 0);
  // steps under way: 16 KB a warp or a little more, 12 warps an SM
  static constexpr int depth = stage >= 8192 ? 2 : 4;
};

}  // namespace

constexpr int kWarps = 4;

template <int D, int kKind, int NB>
__global__ void __launch_bounds__(kWarps * 32, NB == 1 ? 3 : 2)
chunk_rows_kernel(const __grid_constant__ ChunkArgs A, const __grid_constant__ ChunkList list,
                  const __grid_constant__ ChunkUnits units) {
  using Y = Layout<D, kKind>;
  constexpr int KCH = D / 16;
  constexpr int R = 8 * NB;
  extern __shared__ __align__(128) unsigned char s_dyn[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  unsigned char (*s_ring)[Y::stage] =
      reinterpret_cast<unsigned char (*)[Y::stage]>(s_dyn + warp * (Y::depth * Y::stage));
  const int gid = lane >> 2, tig = lane & 3;
  const int total = units.base[list.n];
  // the heads of one part side by side: their rows lie together, and their scales share sectors
  const int c = blockIdx.x / (A.g.H * A.nl), lh = blockIdx.x - c * (A.g.H * A.nl);
  const int h = lh % A.g.H, li = lh / A.g.H;
  const int64_t unit = static_cast<int64_t>(lh) * total + c;
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
  constexpr int kStep = Y::step, kHop = kWarps * Y::step;
  const int v1 = min((split + 1) * A.span, n_vis);
  const int v0 = split * A.span + warp * kStep;      // this warp's first step

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

  pdl_wait();     // (above, the kernel's own arguments only)
  auto position = [&](int v) { return v < sinks ? v : lo + v - sinks; };
  // lane l reads the table for the position of index v + l (16 positions a step: lanes l and
  // l + 16 the same), ahead of its use; the page row is made from it when the copies start
  constexpr uint32_t kAll = kStep == 32 ? 0xFFFFFFFFu : 0xFFFFu;
  int ref_page = -1, ref_slot = 0;
  auto look_up = [&](int v) {
    const int pos = position(min(v + (lane & (kStep - 1)), v1 - 1));
    const int lp = P.p_shift >= 0 ? (pos >> P.p_shift) : pos / P.P;
    ref_slot = pos - lp * P.P;
    ref_page = -1;
    if (lp < P.max_lp) ref_page = __ldg(P.bt + static_cast<int64_t>(list.agent[x]) * P.max_lp + lp);
  };
  // starts the copies of the step at v (looked up before); returns its mapped positions' bits
  const uint32_t ring = smem_u32(s_ring);   // (128-byte aligned: V's rows are swizzled in it)
  const uint8_t* klane = kbase + tig * 16;
  const uint8_t* vlane = vbase + gid * Y::vBytes;
  auto start_copies = [&](int v, int slot) {
    const bool in = v + (lane & (kStep - 1)) < v1;
    const bool mapped = in && ref_page >= 0 && ref_page < P.num_pages;
    const uint32_t have = __ballot_sync(0xFFFFFFFFu, mapped) & kAll;
    const int mine = mapped ? ref_page * P.P + ref_slot : 0;
    if (in && !mapped) atomicOr(A.err, err_bit(TD_ERR_UNMAPPED_PAGE));
    const uint32_t base = ring + slot * Y::stage;
    if constexpr (Y::k8) {
      const uint32_t sc = base + Y::codes + lane * 4;
      copy4(sc, kscale + static_cast<int64_t>(mine) * A.g.H, mapped);
      copy4(sc + kStep * 4, vscale + static_cast<int64_t>(mine) * A.g.H, mapped);
    }
#pragma unroll
    for (int sub = 0; sub < Y::subs; ++sub) {
      const uint32_t dk = base + sub * (Y::kBytes + Y::vAll) + lane * 16;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int at = sub * 16 + gid + 8 * i;
        const int row = __shfl_sync(0xFFFFFFFFu, mine, at);
        const uint8_t* src = klane + static_cast<int64_t>(row) * row_bytes;
        const bool live = (have >> at) & 1u;
#pragma unroll
        for (int j = 0; j < Y::kChunks; ++j)
          copy16(dk + (i * Y::kChunks + j) * 512, src + j * 64, live);
      }
      const uint32_t dv = base + sub * (Y::kBytes + Y::vAll) + Y::kBytes + lane * Y::vBytes;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int at = sub * 16 + 2 * tig + (i & 1) + 8 * (i >> 1);
        const int row = __shfl_sync(0xFFFFFFFFu, mine, at);
        const uint8_t* src = vlane + static_cast<int64_t>(row) * row_bytes;
        const bool live = (have >> at) & 1u;
#pragma unroll
        for (int j = 0; j < Y::vChunks; ++j) {
          const uint32_t to = dv + (i * Y::vChunks + j) * (Y::vBytes * 32);
          if constexpr (!Y::k8) {
            copy16(to ^ ((i & 1) << 6), src + j * 128, live);
          } else if constexpr (Y::vBytes == 16) {
            copy16(to, src + j * 128, live);
          } else {
            // 8 neighbouring codes (D = 64)
            asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(to), "l"(src),
                         "r"(live ? 8 : 0)
                         : "memory");
          }
        }
      }
    }
    return have;
  };

  // the ring: the copies of the first steps start before anything else is loaded
  uint32_t bits[Y::depth];      // mapped positions of the steps in the ring, the oldest first
  if (v0 < v1) look_up(v0);
#pragma unroll
  for (int i = 0; i < Y::depth - 1; ++i) {
    bits[i] = 0;
    if (v0 + i * kHop < v1) {
      bits[i] = start_copies(v0 + i * kHop, i);
      look_up(v0 + (i + 1) * kHop);
    }
    cp_async_commit();
  }
  pdl_trigger();

  // this lane's query rows: as a B-operand column (gid), and as accumulator columns
  int pos_q[NB][2];          // positions of columns 2 tig, 2 tig + 1; -1 past the last row
  uint32_t qf[NB][KCH][2];
  [[maybe_unused]] float row_scale[NB][2];   // 8-bit pages: scale * log2(e) of the columns
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
    if constexpr (Y::k8) {       // f16 fragments, the row's factor kept for its scores
      uint32_t m = 0;
#pragma unroll
      for (int kc = 0; kc < KCH; ++kc)
        m = __vmaxu2(m, __vmaxu2(qf[nb][kc][0] & 0x7FFF7FFFu, qf[nb][kc][1] & 0x7FFF7FFFu));
      m = __vmaxu2(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
      m = __vmaxu2(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
      float inverse;
      const float f = f16_scale(max(m & 0xFFFFu, m >> 16), &inverse);
#pragma unroll
      for (int kc = 0; kc < KCH; ++kc)
#pragma unroll
        for (int e = 0; e < 2; ++e)
          qf[nb][kc][e] = pack_f16(bf_lo(qf[nb][kc][e]) * f, bf_hi(qf[nb][kc][e]) * f);
#pragma unroll
      for (int e = 0; e < 2; ++e)      // (row c's is in the lanes 4 c .. 4 c + 3)
        row_scale[nb][e] = __shfl_sync(0xFFFFFFFFu, inverse, (2 * tig + e) * 4) * A.scale_log2;
    }
  }

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

  int slot = 0;
  for (int v = v0; v < v1; v += kHop) {
    {
      const int ahead = v + (Y::depth - 1) * kHop;
      const int into = slot == 0 ? Y::depth - 1 : slot - 1;
      uint32_t b = 0;
      __syncwarp();                          // the slot has been read by all lanes
      if (ahead < v1) {
        b = start_copies(ahead, into);
        look_up(ahead + kHop);
      }
      cp_async_commit();
      bits[Y::depth - 1] = b;
    }
    cp_async_wait<Y::depth - 1>();
    __syncwarp();                            // scales and bf16 V: the other lanes' copies too
    const uint32_t have = bits[0];
    const unsigned char* st = s_ring[slot];
    const float* scales = reinterpret_cast<const float*>(st + Y::codes);
    // scores: s[sub][nb][i] of position sub * 16 + gid + 8 * (i >> 1), column 2 tig + (i & 1)
    float s[Y::subs][NB][4];
#pragma unroll
    for (int sub = 0; sub < Y::subs; ++sub) {
      const unsigned char* sk = st + sub * (Y::kBytes + Y::vAll) + lane * 16;
      uint4 kr[2][Y::kChunks];               // rows gid, gid + 8
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < Y::kChunks; ++j)
          kr[i][j] = *reinterpret_cast<const uint4*>(sk + (i * Y::kChunks + j) * 512);
      float s2[NB][4];                       // every other product: two chains
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int i = 0; i < 4; ++i) s[sub][nb][i] = s2[nb][i] = 0.0f;
#pragma unroll
      for (int kc = 0; kc < KCH; ++kc) {
        uint32_t a[4];
        if constexpr (Y::k8) {
          const int j = kc >> 2;
          const uint32_t w0 = reinterpret_cast<const uint32_t*>(&kr[0][j])[kc & 3];
          const uint32_t w1 = reinterpret_cast<const uint32_t*>(&kr[1][j])[kc & 3];
          a[0] = word_f16<kKind, false>(w0);
          a[1] = word_f16<kKind, false>(w1);
          a[2] = word_f16<kKind, true>(w0);
          a[3] = word_f16<kKind, true>(w1);
        } else {
          const uint32_t* w0 = reinterpret_cast<const uint32_t*>(&kr[0][kc >> 1]) + (kc & 1) * 2;
          const uint32_t* w1 = reinterpret_cast<const uint32_t*>(&kr[1][kc >> 1]) + (kc & 1) * 2;
          a[0] = w0[0];
          a[1] = w1[0];
          a[2] = w0[1];
          a[3] = w1[1];
        }
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          float* d = kc & 1 ? s2[nb] : s[sub][nb];
          if constexpr (Y::k8) mma_f16(d, a[0], a[1], a[2], a[3], qf[nb][kc][0], qf[nb][kc][1]);
          else mma_bf16(d, a[0], a[1], a[2], a[3], qf[nb][kc][0], qf[nb][kc][1]);
        }
      }
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int i = 0; i < 4; ++i) s[sub][nb][i] = __fadd_rn(s[sub][nb][i], s2[nb][i]);
    }
    // does every row of the tile see every position of the step?
    const int pa = position(v), pb = position(v + kStep - 1);
    const bool whole = have == kAll && pb <= p_first &&
                       (A.window == 0 || pa > p_last - A.window || v + kStep <= sinks);
#pragma unroll
    for (int sub = 0; sub < Y::subs; ++sub) {
      [[maybe_unused]] float ks[2];      // rows gid, gid + 8
      if constexpr (Y::k8) {
        ks[0] = scales[sub * 16 + gid];
        ks[1] = scales[sub * 16 + gid + 8];
      }
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          // (the query row's factor, then K's scale: the two multiplied first could pass float32,
          // and a score of 0 become infinity times 0)
          s[sub][nb][i] = Y::k8 ? __fmul_rn(__fmul_rn(s[sub][nb][i], row_scale[nb][i & 1]), ks[i >> 1])
                                : __fmul_rn(s[sub][nb][i], A.scale_log2);
      if (!whole) {
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int at = sub * 16 + gid + 8 * (i >> 1);
            const int pq = pos_q[nb][i & 1], pp = position(v + at);
            const bool ok = ((have >> at) & 1u) && pp <= pq &&
                            (A.window == 0 || pp > pq - A.window || pp < A.n_sink);
            // (-infinity says out of sight below, so a score that is -infinity by itself becomes
            // the least number; a bit a score in a register cost 1.7% of an int8 token's time)
            s[sub][nb][i] = ok ? max_nan(s[sub][nb][i], -3.402823466e38f) : -INFINITY;
          }
      }
    }
    // the weights, in base 2 under the running maximum
    float fac[NB][2], w[Y::subs][NB][4];
    bool grew = false;
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float mx = fmaxf(s[0][nb][e], s[0][nb][e + 2]);
        if constexpr (Y::subs == 2) mx = fmaxf(mx, fmaxf(s[1][nb][e], s[1][nb][e + 2]));
        mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 4));
        mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 8));
        mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 16));
        const float m_new = fmaxf(m_run[nb][e], mx);
        // (nothing seen so far: -infinity minus 0, so that the weights come out 0)
        const float sub0 = m_new == -INFINITY ? 0.0f : m_new;
        fac[nb][e] = ex2(__fsub_rn(m_run[nb][e], sub0));
        grew |= m_new != m_run[nb][e];
        m_run[nb][e] = m_new;
        float sum = 0.0f;
#pragma unroll
        for (int sub = 0; sub < Y::subs; ++sub)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            w[sub][nb][e + 2 * i] = ex2(__fsub_rn(s[sub][nb][e + 2 * i], sub0));
            sum = __fadd_rn(sum, w[sub][nb][e + 2 * i]);
          }
        l_part[nb][e] = __fmaf_rn(l_part[nb][e], fac[nb][e], sum);
      }
    if (__any_sync(0xFFFFFFFFu, grew)) {
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int mt = 0; mt < KCH; ++mt) {
          acc[nb][mt][0] *= fac[nb][0];
          acc[nb][mt][1] *= fac[nb][1];
          acc[nb][mt][2] *= fac[nb][0];
          acc[nb][mt][3] *= fac[nb][1];
        }
    }
#pragma unroll
    for (int sub = 0; sub < Y::subs; ++sub) {
      // p: the weight on V, with the row's scale
      float p[NB][4];
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int i = 0; i < 4; ++i) p[nb][i] = w[sub][nb][i];
      if constexpr (Y::k8) {
        const float vs[2] = {scales[kStep + sub * 16 + gid], scales[kStep + sub * 16 + gid + 8]};
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            p[nb][i] = __fmul_rn(p[nb][i], vs[i >> 1]);
            // (a position out of sight keeps the weight 0 whatever its scale)
            if (!whole && s[sub][nb][i] == -INFINITY) p[nb][i] = 0.0f;
          }
      }
      const unsigned char* sv = st + sub * (Y::kBytes + Y::vAll) + Y::kBytes;
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
      if constexpr (!Y::k8) {
        // element (position k, dim d) of V in the ring
        auto v_at = [&](int k, int d) {
          const int i = (k & 1) + 2 * (k >> 3), ch = d >> 3;
          return const_cast<unsigned char*>(sv) + (i * Y::vChunks + (ch >> 3)) * 512 +
                 ((((ch & 7) * 4 + ((k & 7) >> 1)) * 16) ^ ((i & 1) << 6)) + (d & 7) * 2;
        };
        // values that must not meet the zero weight of a row out of whose sight they are (rare: a
        // step that masks, with such a value): their terms are added to the rows that see them,
        // under whatever weight (0 times a NaN or an infinity is a NaN, as in a step that masks
        // nothing), and they leave the product
        if (!whole) {
          bool bad = false;
#pragma unroll
          for (int i = 0; i < 4 * Y::vChunks; ++i) {
            const uint4 q4 = *reinterpret_cast<const uint4*>(sv + i * 512 + lane * 16);
            bad |= nonfinite2(q4.x) || nonfinite2(q4.y) || nonfinite2(q4.z) || nonfinite2(q4.w);
          }
          if (__any_sync(0xFFFFFFFFu, bad)) {
#pragma unroll 1
            for (int k = 0; k < 16; ++k) {
              float pk[NB][2];
              bool sees[NB][2];
#pragma unroll
              for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                  const float mine = k < 8 ? p[nb][e] : p[nb][e + 2];
                  pk[nb][e] = __shfl_sync(0xFFFFFFFFu, mine, (k & 7) * 4 + tig);
                  const float score = k < 8 ? s[sub][nb][e] : s[sub][nb][e + 2];
                  sees[nb][e] = __shfl_sync(0xFFFFFFFFu, score, (k & 7) * 4 + tig) != -INFINITY;
                }
#pragma unroll
              for (int mt = 0; mt < KCH; ++mt)
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                  const uint32_t b =
                      *reinterpret_cast<const uint16_t*>(v_at(k, mt * 16 + half * 8 + gid));
                  if ((b & 0x7F80u) != 0x7F80u) continue;
#pragma unroll
                  for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                    for (int e = 0; e < 2; ++e)
                      if (sees[nb][e])
                        acc[nb][mt][half * 2 + e] =
                            __fmaf_rn(pk[nb][e], __uint_as_float(b << 16), acc[nb][mt][half * 2 + e]);
                }
            }
            __syncwarp();
            uint16_t* mine = reinterpret_cast<uint16_t*>(const_cast<unsigned char*>(sv)) + lane * 8;
#pragma unroll 1
            for (int i = 0; i < 4 * Y::vChunks * 8; ++i) {
              uint16_t* at = mine + (i >> 3) * 256 + (i & 7);
              if ((*at & 0x7F80u) == 0x7F80u) *at = 0;
            }
            __syncwarp();
          }
        }
        // V^T's fragments: dims as rows, transposed as they are read. Lane l names a row of 8
        // dims: position (l & 7) + 8 (l >> 4), dims 16 mt + 8 ((l >> 3) & 1)
        const uint32_t v0a = smem_u32(v_at((lane & 7) + 8 * (lane >> 4), 8 * ((lane >> 3) & 1)));
#pragma unroll
        for (int mt = 0; mt < KCH; ++mt) {
          uint32_t a[4];
          // 16 dims are two vectors on: 128 bytes, 512 for every 64 dims
          ldmatrix_x4_trans(a, v0a + (mt >> 2) * 512 + (mt & 3) * 128);
#pragma unroll
          for (int nb = 0; nb < NB; ++nb) {
            mma_bf16(acc[nb][mt], a[0], a[1], a[2], a[3], ph[nb][0], ph[nb][1]);
            mma_bf16(acc[nb][mt], a[0], a[1], a[2], a[3], pl[nb][0], pl[nb][1]);
          }
        }
      } else {
        uint32_t vr[4][Y::vWords];   // rows 2 tig, 2 tig + 1, 2 tig + 8, 2 tig + 9
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const unsigned char* at = sv + lane * Y::vBytes + i * (Y::vBytes * 32);
          if constexpr (Y::vBytes == 16) {
            const uint4 q4 = *reinterpret_cast<const uint4*>(at);
            vr[i][0] = q4.x;
            vr[i][1] = q4.y;
            vr[i][2] = q4.z;
            vr[i][3] = q4.w;
          } else {
            const uint2 q2 = *reinterpret_cast<const uint2*>(at);
            vr[i][0] = q2.x;
            vr[i][1] = q2.y;
          }
        }
#pragma unroll
        for (int mt = 0; mt < KCH; ++mt) {
          const int w8 = mt >> 1, i0 = (mt & 1) * 2;   // word and first byte of dims 2 mt, 2 mt + 1
          const uint32_t a0 = pair_bf16<kKind>(vr[0][w8], vr[1][w8], i0);
          const uint32_t a1 = pair_bf16<kKind>(vr[0][w8], vr[1][w8], i0 + 1);
          const uint32_t a2 = pair_bf16<kKind>(vr[2][w8], vr[3][w8], i0);
          const uint32_t a3 = pair_bf16<kKind>(vr[2][w8], vr[3][w8], i0 + 1);
#pragma unroll
          for (int nb = 0; nb < NB; ++nb) {
            mma_bf16(acc[nb][mt], a0, a1, a2, a3, ph[nb][0], ph[nb][1]);
            mma_bf16(acc[nb][mt], a0, a1, a2, a3, pl[nb][0], pl[nb][1]);
          }
        }
      }
    }
#pragma unroll
    for (int i = 0; i + 1 < Y::depth; ++i) bits[i] = bits[i + 1];
    slot = slot + 1 == Y::depth ? 0 : slot + 1;
  }

  // The warps' results joined. The lane's dims of acc[mt]: bf16 16 mt + gid and 16 mt + gid + 8;
  // 8-bit gid vDims + 2 mt and the next one.
  constexpr int kLd = D + 4;                       // floats per row: a quad's rows 8 banks apart
  float* s_o = reinterpret_cast<float*>(s_dyn);    // [kWarps][R][kLd], over the rings
  __shared__ float s_m[kWarps][R], s_l[kWarps][R];
  cp_async_wait<0>();
#pragma unroll
  for (int nb = 0; nb < NB; ++nb)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float l = l_part[nb][e];
      l += __shfl_xor_sync(0xFFFFFFFFu, l, 4);
      l += __shfl_xor_sync(0xFFFFFFFFu, l, 8);
      l += __shfl_xor_sync(0xFFFFFFFFu, l, 16);
      if (gid == 0) {
        s_m[warp][nb * 8 + 2 * tig + e] = m_run[nb][e];
        s_l[warp][nb * 8 + 2 * tig + e] = l;
      }
    }
  __syncthreads();                                 // (and no ring is read any more)
#pragma unroll
  for (int nb = 0; nb < NB; ++nb)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int rt = nb * 8 + 2 * tig + e;
      const float top = fmaxf(fmaxf(s_m[0][rt], s_m[1][rt]), fmaxf(s_m[2][rt], s_m[3][rt]));
      const float f = ex2(__fsub_rn(m_run[nb][e], top == -INFINITY ? 0.0f : top));
      float* o = s_o + (warp * R + rt) * kLd;
#pragma unroll
      for (int mt = 0; mt < KCH; ++mt) {
        if constexpr (Y::k8) {
          *reinterpret_cast<float2*>(o + gid * Y::vDims + 2 * mt) =
              make_float2(acc[nb][mt][e] * f, acc[nb][mt][2 + e] * f);
        } else {
          o[mt * 16 + gid] = acc[nb][mt][e] * f;
          o[mt * 16 + gid + 8] = acc[nb][mt][2 + e] * f;
        }
      }
    }
  __syncthreads();
  // 8 dims a thread
  for (int i = threadIdx.x; i < R * (D / 8); i += kWarps * 32) {
    const int rt = i / (D / 8), d = (i % (D / 8)) * 8;
    const int r = r0 + rt;
    if (r >= rows) continue;
    const float top = fmaxf(fmaxf(s_m[0][rt], s_m[1][rt]), fmaxf(s_m[2][rt], s_m[3][rt]));
    float l = 0.0f, y[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) y[k] = 0.0f;
#pragma unroll
    for (int wp = 0; wp < kWarps; ++wp) {
      l = __fmaf_rn(s_l[wp][rt], ex2(__fsub_rn(s_m[wp][rt], top == -INFINITY ? 0.0f : top)), l);
      const float* o = s_o + (wp * R + rt) * kLd + d;
#pragma unroll
      for (int k = 0; k < 8; k += 4) {
        const float4 q4 = *reinterpret_cast<const float4*>(o + k);
        y[k] += q4.x;
        y[k + 1] += q4.y;
        y[k + 2] += q4.z;
        y[k + 3] += q4.w;
      }
    }
    if (A.direct) {
      const int tok = r / A.G;
      const int64_t row = (static_cast<int64_t>(li) * A.tokens + list.tok[x] + tok) * A.nq +
                          h * A.G + (r - tok * A.G);
      const float inv = l == 0.0f ? 0.0f : 1.0f / l;      // a row that sees nothing: zeros
#pragma unroll
      for (int k = 0; k < 8; ++k) y[k] *= inv;
      st16(A.out + row * D + d, pack8(y));
      if (d == 0 && A.lse)
        A.lse[row] = l == 0.0f ? -INFINITY : (top + log2f(l)) * 0.69314718055994530942f;
    } else {
      float* po = A.part_o + (unit * R + rt) * D + d;
#pragma unroll
      for (int k = 0; k < 8; k += 4)
        *reinterpret_cast<float4*>(po + k) = make_float4(y[k], y[k + 1], y[k + 2], y[k + 3]);
      if (d == 0) {
        A.part_ml[(unit * R + rt) * 2] = top;
        A.part_ml[(unit * R + rt) * 2 + 1] = l;
      }
    }
  }
}

// The parts of every (layer, token, query head) row joined. kSplit: a CTA of four warps a row,
// warp w taking parts w, w + 4, ..., their loads all under way together (few rows: latency);
// else a warp a row, four rows a CTA (many rows: bandwidth). A part that saw nothing has the
// maximum -inf, and is not used. A row's place is found before the previous kernel has ended,
// and the first parts are loaded beside their maxima (one after the other: 27.7 us against 26.2
// for a token of 10 agents, 3.5 of which were the join).
constexpr int kJoinWarps = 4;

template <int D, bool kSplit>
__global__ void __launch_bounds__(kJoinWarps * 32)
chunk_join_kernel(const __grid_constant__ ChunkArgs A, const __grid_constant__ ChunkList list,
                  const __grid_constant__ ChunkUnits units, int R) {
  constexpr int DPL = D / 32;
  __shared__ float s_acc[kJoinWarps][D];
  __shared__ float s_l[kJoinWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int n_tok = list.row[list.n] - A.join_from;
  const unsigned n = kSplit ? blockIdx.x : blockIdx.x * kJoinWarps + warp;
  const int gq = static_cast<int>(n % A.nq);
  const int lt = static_cast<int>(n / A.nq);
  if (!kSplit && lt >= A.nl * n_tok) return pdl_wait();
  const int t = A.join_from + lt % n_tok, li = lt / n_tok;
  int x = 0;
  for (int hi = list.n - 1; x < hi;) {
    const int mid = (x + hi + 1) >> 1;
    if (list.row[mid] <= t) x = mid;
    else hi = mid - 1;
  }
  const int h = gq / A.G;
  const int r = (t - list.row[x]) * A.G + gq - h * A.G;
  const int tile = r / R, rt = r - tile * R;
  const int ns = units.nsplit[x], whole = units.whole[x];
  // (the tensor-core kernel, whose tiles are larger, numbers them from the last one down)
  const int at = R < 128 ? tile : ((list.row[x + 1] - list.row[x]) * A.G - 1) / R - tile;
  if (at < whole) return pdl_wait();              // written already
  const int64_t u0 =
      (static_cast<int64_t>(li) * A.g.H + h) * (units.base[list.n] - A.whole_units) +
      (units.base[x] + whole - A.whole_units) + static_cast<int64_t>(at - whole) * ns;
  pdl_wait();     // (above, the kernel's own arguments only)
  // this warp's first parts, on their way while the maximum is found (those that saw nothing
  // hold anything, and are not used)
  constexpr int kFirst = 4, kHop = kSplit ? kJoinWarps : 1;
  const int i0 = kSplit ? warp : 0;
  auto load = [&](int i, float2* ml, float* q) {
    const int64_t pr = (u0 + i) * R + rt;
    *ml = *reinterpret_cast<const float2*>(A.part_ml + pr * 2);
    const float* po = A.part_o + pr * D + lane * DPL;
    if constexpr (DPL == 4) {
      const float4 f = *reinterpret_cast<const float4*>(po);
      q[0] = f.x;
      q[1] = f.y;
      q[2] = f.z;
      q[3] = f.w;
    } else {
      const float2 f = *reinterpret_cast<const float2*>(po);
      q[0] = f.x;
      q[1] = f.y;
    }
  };
  float2 ml0[kFirst];
  float q0[kFirst][DPL];
#pragma unroll
  for (int u = 0; u < kFirst; ++u) {
    ml0[u] = make_float2(-INFINITY, 0.0f);
    if (i0 + u * kHop < ns) load(i0 + u * kHop, &ml0[u], q0[u]);
  }
  // every warp finds the row's maximum itself
  float mx = -INFINITY;
  bool nan = false;
  for (int i = lane; i < ns; i += 32) {
    const float2 ml = *reinterpret_cast<const float2*>(A.part_ml + ((u0 + i) * R + rt) * 2);
    mx = fmaxf(mx, ml.x);
    nan |= ml.y != ml.y;      // scores that are NaN leave the maximum and make the sum NaN
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, o));
  float l = 0.0f, acc[DPL];
#pragma unroll
  for (int d = 0; d < DPL; ++d) acc[d] = 0.0f;
  auto add = [&](const float2& ml, const float* q) {
    if (ml.x == -INFINITY) return;
    const float w = exp2f(ml.x - mx);
    l = __fmaf_rn(ml.y, w, l);
#pragma unroll
    for (int d = 0; d < DPL; ++d) acc[d] = __fmaf_rn(q[d], w, acc[d]);
  };
#pragma unroll
  for (int u = 0; u < kFirst; ++u) add(ml0[u], q0[u]);
#pragma unroll 4
  for (int i = i0 + kFirst * kHop; i < ns; i += kHop) {
    float2 ml;
    float q[DPL];
    load(i, &ml, q);
    add(ml, q);
  }
  nan = __any_sync(0xFFFFFFFFu, nan);
  if constexpr (kSplit) {
#pragma unroll
    for (int d = 0; d < DPL; ++d) s_acc[warp][lane * DPL + d] = acc[d];
    if (lane == 0) s_l[warp] = l;
    __syncthreads();
    if (warp != 0) return;
    l = (s_l[0] + s_l[1]) + (s_l[2] + s_l[3]);
#pragma unroll
    for (int d = 0; d < DPL; ++d) {
      const int c = lane * DPL + d;
      acc[d] = (s_acc[0][c] + s_acc[1][c]) + (s_acc[2][c] + s_acc[3][c]);
    }
  }
  if (nan) l = __uint_as_float(0x7FC00000u);
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
                            int rows_per_tile, bool fresh, cudaStream_t st) {
  const int64_t n = static_cast<int64_t>(a.nl) * a.g.H * units.base[list.n];
  if (n == 0) return cudaSuccess;
  const unsigned grid = static_cast<unsigned>(n);
  using Y = Layout<D, kKind>;
  constexpr int kSmem = kWarps * Y::depth * Y::stage;
  static_assert(kSmem >= kWarps * 16 * (D + 4) * 4, "the rings' space takes the warps' results");
  auto* kernel = rows_per_tile == 8 ? chunk_rows_kernel<D, kKind, 1> : chunk_rows_kernel<D, kKind, 2>;
  if (fresh) {
    const cudaError_t e =
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess) return e;
  }
  return launch_after(kernel, grid, kWarps * 32, kSmem, st, a, list, units);
}

cudaError_t launch_chunk_rows(const ChunkArgs& a, const ChunkList& list, const ChunkUnits& units,
                              CacheKind kind, int rows_per_tile, bool fresh, cudaStream_t st) {
  if (a.g.D != 64 && a.g.D != 128) return cudaErrorInvalidValue;
  const bool wide = a.g.D == 128;
  switch (kind) {
    case kCacheBf16:
      return wide ? run_rows<128, kCacheBf16>(a, list, units, rows_per_tile, fresh, st)
                  : run_rows<64, kCacheBf16>(a, list, units, rows_per_tile, fresh, st);
    case kCacheInt8:
      return wide ? run_rows<128, kCacheInt8>(a, list, units, rows_per_tile, fresh, st)
                  : run_rows<64, kCacheInt8>(a, list, units, rows_per_tile, fresh, st);
    case kCacheE4m3:
      return wide ? run_rows<128, kCacheE4m3>(a, list, units, rows_per_tile, fresh, st)
                  : run_rows<64, kCacheE4m3>(a, list, units, rows_per_tile, fresh, st);
  }
  return cudaErrorInvalidValue;
}

cudaError_t launch_chunk_join(const ChunkArgs& a, const ChunkList& list, const ChunkUnits& units,
                              int rows_per_tile, cudaStream_t st) {
  const unsigned rows = static_cast<unsigned>(a.nl) * (list.row[list.n] - a.join_from) * a.nq;
  // a warp a row from 8192 rows on (the machine holds 152 x 64 warps)
  const bool split = rows < 8192;
  const unsigned grid = split ? rows : (rows + kJoinWarps - 1) / kJoinWarps;
  auto* wide = split ? chunk_join_kernel<128, true> : chunk_join_kernel<128, false>;
  auto* narrow = split ? chunk_join_kernel<64, true> : chunk_join_kernel<64, false>;
  return launch_after(a.g.D == 128 ? wide : narrow, grid, kJoinWarps * 32, 0, st, a, list, units,
                      rows_per_tile);
}

}  // namespace td
