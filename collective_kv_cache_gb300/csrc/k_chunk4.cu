// k_chunk4.cu - attention over 4-bit pages for a few query rows: chunks of a few tokens (their
// batch from the host), and one token a request (the lengths read on the device).
//
// The mathematics is k_chunk.cu's: a token at pos sees p <= pos (under a window W p > pos - W or
// p < n_sink); out = softmax(scale q . k_p) v_p over what it sees. A block takes units = (layer, kv
// head, tile of 8 or 16 query rows, a part of the tile's visible positions), its four warps every
// fourth step of 32 positions; products are mma.sync m16n8k16 with positions or dims as the 16 rows
// and query rows as the columns. What is different is the operands:
//   int4   a code u of 0 to 15 in the low bits of a 16-bit half is the f16 subnormal u 2^-24, and four
//          bits higher 16 u 2^-24: a mask makes two operands of a word, without a conversion (a
//          shift by 8 brings the other half of the codes there). The queries' elements that meet the
//          higher ones are a sixteenth, the outputs of such dims are divided by 16. The zero point z
//          comes off the sums: sum q (u - z) = sum q u - z sum q in float32, sum p (u - z) = sum p u -
//          sum p z by one product more, where z is such an operand too. (The tensor cores cut addends
//          some 24 bits below the largest, a subnormal's counted as 2^-14: bits that q's elements, of 8,
//          leave free and their sum does not. With z times the sum a product too, of three f16 parts, the
//          log-sum-exp of a few positions was 1e-5 to 3e-5 off; 2e-6 to 3e-6 so, and the call 2% faster.)
//   e2m1   two codes a conversion instruction. K's quarters are products of their own, each under its
//          power of two; V's elements take that of their quarter relative to the row's largest, which
//          goes on the weight.
// Everything is f16: the queries, each row under a power of two (64 to 128 the largest element), and
// the weights times V's scales, under a power of two that the warp keeps (2^6 over that of the largest
// scale so far), so one product does where bf16 weights of 16 bits take two. The reference of the
// weights is lazy: raised to the maximum only when that has passed it by 2^8, so most steps take a
// vote instead of an exchange.
//
// Steps come through a ring of cp.async copies as in k_chunk.cu, rows as they lie in the page but for
// the order of their 16-byte pieces (piece_at), and are read back as fragments; int4's V, where pairs
// of positions make an operand, by transposing loads.
//
// All sequences' steps of 128 positions lie end to end, and every block of a (layer, kv head) takes the
// same number of them, whichever sequences they belong to; where few are taken, blocks end with
// their sequence instead (Cut). A tile's parts are joined by a kernel of their own. (The last block of a
// tile joining them itself: a step of 10 agents 16.8 us and 15.4 so.)
//
// Measured on one GB300, 4 kv heads of 7 query heads, D = 128: one token of 64 requests on 8192 to 24576
// positions 105 us over int4 pages (5.5 TB/s; the copies alone take 95), 115 over e2m1 (5.0); at D = 64
// 76 and 81. Two tokens each on 4096 to 12288: 78 and 85 us, tensor pipe 38% and issue slots 46% busy: 12
// warps an SM wait for their own products and shared memory in turn. Ten requests on 3060 to 6560 15.5
// us, of which 14.3 remain in a graph.
#include "td_cache4.cuh"
#include "td_cache8.cuh"

namespace td {

namespace {

constexpr int kWarps = 4;
constexpr int kStep = 32;                 // positions a warp's step
constexpr int kHop = kWarps * kStep;      // and the block's
constexpr float kLazy = 8.0f;             // the reference lags the maximum by this much at most (base 2)

__device__ __forceinline__ void mma_f16(float* d, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, "
      "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// The first product of a sum.
__device__ __forceinline__ void mma_f16_new(float* d, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, "
      "{%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.0f));
}
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
// 16 (4) bytes into shared memory; zeros where `live` is not set.
template <bool kAll>
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool live) {
  if constexpr (kAll)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
  else
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
                 "r"(live ? 16 : 0)
                 : "memory");
}
__device__ __forceinline__ void copy4(uint32_t dst, const void* src, bool live) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src),
               "r"(live ? 4 : 0)
               : "memory");
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

struct Always {
  static constexpr bool value = true;
};
struct Maybe {
  static constexpr bool value = false;
};

template <int D, int kKind>
struct Ring {
  static constexpr int kRow = D / 2;                    // bytes of a row of codes
  static constexpr int kCh = kRow / 16;                 // ... and 16-byte pieces
  static constexpr int kCodes = kStep * kRow;           // of a step's K or V
  static constexpr int kStage = 2 * kCodes + 2 * kStep * 4;
  static constexpr int kDepth = D == 128 ? 3 : 4;
  // e2m1: of a step, the scales of K's quarters, V's quarters' factors and V's scales
  static constexpr int kFacts = kKind == kCacheE2m1 ? kStep * (16 + 8 + 4) : 0;
  static constexpr int kWarp = kDepth * kStage + kFacts;
  static constexpr int kRings = kWarps * kWarp;
  // then, with 16 rows a tile, the queries' fragments (in registers they left room for two blocks an
  // SM instead of three)
  static constexpr int kQueries = (D / 16) * 2 * 32 * 8;
  static constexpr int smem(int rows) { return kRings + (rows == 16 ? kQueries : 0); }
};

// Byte offset of 16-byte piece c of position r's row: eight rows' pieces of one number lie in eight
// different places of 128 bytes.
template <int D>
__device__ __forceinline__ int piece_at(int r, int c) {
  return r * (D / 2) + (D == 128 ? c ^ ((r >> 1) & 3) : c ^ ((r >> 2) & 1)) * 16;
}
// The position (of 16) that is row r of a product. e2m1 reads V's rows 2 tig and 2 tig + 1 by 8 (4)
// bytes a lane: with the low bits mixed so they meet every bank once.
template <int D, bool kInt4>
__device__ __forceinline__ int position16(int r) {
  if constexpr (kInt4) return r;
  return D == 128 ? r ^ ((r >> 1) & 1) : r ^ ((r >> 2) & 1);
}
// Four 8 x 8 matrices of 16-bit values, transposed: lane l names row l & 7 of matrix l >> 3.
__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t* r, uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

// A unit: a part of a tile's positions. In shared memory: what is needed at the end only is read
// again there (kept in registers over the loop it was spilled).
struct Place {
  int agent;                // row of the block table
  int start, len;           // position of the sequence's first token, and its tokens
  int tok;                  // dense row of that token
  int tile;
  int v_begin, v_end;       // the part: visible positions, by number
  int64_t unit;             // number of its partial results
  int direct;               // it has all of the tile's positions, and writes the outputs
  int64_t left;             // steps that the block has left, this unit's included
  int x, n;                 // sequence, steps of the unit
};

template <int D, int kKind, int NB>
__device__ __forceinline__ void attend(const ChunkArgs& A, const volatile Place& w,
                                       unsigned char* s_dyn) {
  using Y = Ring<D, kKind>;
  constexpr bool kInt4 = kKind == kCacheInt4;
  constexpr int KCH = D / 16, R = 8 * NB;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int gid = lane >> 2, tig = lane & 3;
  const int lh = static_cast<int>(blockIdx.x % static_cast<unsigned>(A.g.H * A.nl));
  const int h = lh % A.g.H, li = lh / A.g.H;
  const int start = w.start, rows = w.len * A.G, r0 = w.tile * R;
  // the tile's visible positions, numbered v: the first `sinks`, then lo .. p_last
  const int p_first = start + r0 / A.G;
  const int p_last = start + min(r0 + R - 1, rows - 1) / A.G;
  const int lo = A.window ? max(0, p_first - A.window + 1) : 0;
  const int sinks = A.window ? min(A.n_sink, lo) : 0;
  const int skip = lo - sinks;                  // v >= sinks is position v + skip
  const int v1 = min(w.v_end, p_last + 1 - skip);
  const int v0 = w.v_begin + warp * kStep;      // this warp's first step

  const PoolDev& P = A.pool;
  const int H = A.g.H;
  const int64_t plane_rows = P.num_pages * P.P * H;
  const int64_t plane = (static_cast<int64_t>(A.layer_begin + li) * 2) * plane_rows;
  const int cp_pos = lane / Y::kCh, cp_piece = lane % Y::kCh;
  const uint32_t cp_to = piece_at<D>(cp_pos, cp_piece);
  const uint8_t* kcodes =
      reinterpret_cast<const uint8_t*>(P.base) + plane * Y::kRow + cp_piece * 16;
  const uint8_t* vcodes = kcodes + plane_rows * Y::kRow;
  const uint32_t* kword = A.word + plane;
  const uint32_t* vword = kword + plane_rows;
  const int32_t* table = P.bt + static_cast<int64_t>(w.agent) * P.max_lp;
  const unsigned num_pages = static_cast<unsigned>(P.num_pages);

  // steps from v_from to v_to are in every row's sight as a whole (those among the first tokens
  // are looked at one by one)
  const int v_from = A.window ? max(sinks, p_last - A.window + 1 - skip) : 0;
  const int v_to = p_first - skip - (kStep - 1);

  auto position = [&](int v) { return v < sinks ? v : v + skip; };
  // lane l reads the table for the position of number v + l, ahead of its use (every position is
  // within the table: the host or token_steps has seen to that)
  int ref_page = -1, ref_slot = 0;
  auto look_up = [&](int v) {
    const int pos = position(min(v + lane, v1 - 1));
    const int lp = P.p_shift >= 0 ? (pos >> P.p_shift) : pos / P.P;
    ref_slot = pos - lp * P.P;
    ref_page = table[lp];
  };
  unsigned char* s_ring = s_dyn + warp * Y::kWarp;
  const uint32_t ring = smem_u32(s_ring);
  // starts the copies of the step at v (looked up before); returns its mapped positions' bits
  auto start_copies = [&](int v, int slot) {
    const bool in = v + lane < v1;
    const bool mapped = in && static_cast<unsigned>(ref_page) < num_pages;
    const uint32_t have = __ballot_sync(0xFFFFFFFFu, mapped);
    const int mine = mapped ? (ref_page * H + h) * P.P + ref_slot : 0;
    const uint32_t base = ring + slot * Y::kStage;
    copy4(base + 2 * Y::kCodes + lane * 4, kword + mine, mapped);
    copy4(base + 2 * Y::kCodes + kStep * 4 + lane * 4, vword + mine, mapped);
    auto rows_of = [&](auto all) {
#pragma unroll
      for (int i = 0; i < Y::kCh; ++i) {
        const int at = i * (32 / Y::kCh) + cp_pos;
        const int row = __shfl_sync(0xFFFFFFFFu, mine, at);
        const bool live = (have >> at) & 1u;
        // (pieces of positions 8 or 16 on lie in the same place of their rows)
        const uint32_t to = base + cp_to + i * (32 / Y::kCh) * Y::kRow;
        copy16<decltype(all)::value>(to, kcodes + static_cast<int64_t>(row) * Y::kRow, live);
        copy16<decltype(all)::value>(to + Y::kCodes, vcodes + static_cast<int64_t>(row) * Y::kRow, live);
      }
    };
    if (have == 0xFFFFFFFFu) {
      rows_of(Always{});
    } else {
      if (in && !mapped) atomicOr(A.err, err_bit(TD_ERR_UNMAPPED_PAGE));
      rows_of(Maybe{});
    }
    return have;
  };

  uint32_t bits[Y::kDepth];     // mapped positions of the steps in the ring, the oldest first
  if (v0 < v1) look_up(v0);
#pragma unroll
  for (int i = 0; i < Y::kDepth - 1; ++i) {
    bits[i] = 0;
    if (v0 + i * kHop < v1) {
      bits[i] = start_copies(v0 + i * kHop, i);
      look_up(v0 + (i + 1) * kHop);
    }
    cp_async_commit();
  }
  pdl_trigger();

  // the query rows: as a B-operand column (gid), and as accumulator columns (2 tig, 2 tig + 1)
  int pos_q[NB][2];             // positions of the columns; -1 past the last row
  constexpr bool kKeep = NB == 1;
  uint2* s_q = reinterpret_cast<uint2*>(s_dyn + Y::kRings) + lane;    // (all warps write the same)
  [[maybe_unused]] uint2 qf[kKeep ? KCH : 1];
  auto query = [&](int nb, int kc) { return kKeep ? qf[kKeep ? kc : 0] : s_q[(nb * KCH + kc) * 32]; };
  float row_scale[NB][2];       // scale * log2(e) under the row's power of two
  [[maybe_unused]] float q_sum[NB][2];          // int4: less the row's sum, 2^-24 of it
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
    const int64_t row = static_cast<int64_t>(li) * A.tokens + w.tok + tok;
    // the dims that the lane's words of K's row hold: int4 a quarter of the row, e2m1 a quarter of
    // each quarter
    const uint16_t* q = A.q + (row * A.nq + h * A.G + (live ? r - tok * A.G : 0)) * D;
    uint4 raw[D / 32];
    if (!live) {
#pragma unroll
      for (int i = 0; i < D / 32; ++i) raw[i] = make_uint4(0u, 0u, 0u, 0u);
    } else if constexpr (kInt4) {
#pragma unroll
      for (int i = 0; i < D / 32; ++i) raw[i] = ldg16(q + tig * (D / 4) + i * 8);
    } else if constexpr (D == 128) {
#pragma unroll
      for (int i = 0; i < 4; ++i) raw[i] = ldg16(q + i * 32 + tig * 8);
    } else {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint2 x = __ldg(reinterpret_cast<const uint2*>(q + 2 * i * 16 + tig * 4));
        const uint2 y = __ldg(reinterpret_cast<const uint2*>(q + (2 * i + 1) * 16 + tig * 4));
        raw[i] = make_uint4(x.x, x.y, y.x, y.y);
      }
    }
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < D / 32; ++i)
      m = __vmaxu2(m, __vmaxu2(__vmaxu2(raw[i].x & 0x7FFF7FFFu, raw[i].y & 0x7FFF7FFFu),
                               __vmaxu2(raw[i].z & 0x7FFF7FFFu, raw[i].w & 0x7FFF7FFFu)));
    m = __vmaxu2(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
    m = __vmaxu2(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
    float inverse;
    const float f = f16_scale(max(m & 0xFFFFu, m >> 16), &inverse) * 0x1p-8f;
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {          // the word of 8 codes: two products
      float x[8];
      unpack8(raw[i], x);
#pragma unroll
      for (int k = 0; k < 8; ++k) x[k] *= f;
      uint2 a, b;
      if constexpr (kInt4) {
        // masks take codes (0, 4), (1, 5) 16 times, then (2, 6), (3, 7)
        a = make_uint2(pack_f16(x[0], x[4]), pack_f16(x[1] * 0.0625f, x[5] * 0.0625f));
        b = make_uint2(pack_f16(x[2], x[6]), pack_f16(x[3] * 0.0625f, x[7] * 0.0625f));
        sum += (f16_lo(a.x) + f16_hi(a.x)) + (f16_lo(b.x) + f16_hi(b.x)) +
               16.0f * ((f16_lo(a.y) + f16_hi(a.y)) + (f16_lo(b.y) + f16_hi(b.y)));
      } else {
        a = make_uint2(pack_f16(x[0], x[1]), pack_f16(x[2], x[3]));
        b = make_uint2(pack_f16(x[4], x[5]), pack_f16(x[6], x[7]));
      }
      if constexpr (kKeep) {
        qf[2 * i] = a;
        qf[2 * i + 1] = b;
      } else {
        s_q[(nb * KCH + 2 * i) * 32] = a;
        s_q[(nb * KCH + 2 * i + 1) * 32] = b;
      }
    }
    if constexpr (kInt4) {
      sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 1);
      sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 2);
    }
#pragma unroll
    for (int e = 0; e < 2; ++e) {               // (row c's is in the lanes 4 c .. 4 c + 3)
      const float inv = __shfl_sync(0xFFFFFFFFu, inverse, (2 * tig + e) * 4);
      // (int4's products come out 2^24 too small)
      row_scale[nb][e] = inv * 0x1p8f * A.scale_log2 * (kInt4 ? 0x1p24f : 1.0f);
      if constexpr (kInt4) q_sum[nb][e] = __shfl_sync(0xFFFFFFFFu, sum, (2 * tig + e) * 4) * -0x1p-24f;
    }
  }

  // O^T: acc[nb][mt] = the lane's dims 2 mt, 2 mt + 1 x rows 2 tig, 2 tig + 1, under the weights'
  // power of two; int4: 2^-24 of it, and 16 times that in the odd dims
  float acc[NB][KCH][4];
  [[maybe_unused]] float z_acc[NB][4];          // int4: the zero points' sums, 2^-24 of them ([0], [1])
  float m_neg[NB][2], l_part[NB][2];            // less the weights' reference (0 while there is none)
  uint32_t top = 15u << 23;                     // power of two of the largest scale of V so far, as
  float under = __uint_as_float(245u << 23);    // bits, and 2^6 over it
  uint32_t unset = 0u;                          // columns without a reference: bit nb * 2 + e
#pragma unroll
  for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      m_neg[nb][e] = 0.0f;
      l_part[nb][e] = 0.0f;
      // (columns past the last row, whose scores are 0, need none)
      if (pos_q[nb][e] >= 0) unset |= 1u << (nb * 2 + e);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (kInt4) z_acc[nb][i] = 0.0f;
#pragma unroll
      for (int mt = 0; mt < KCH; ++mt) acc[nb][mt][i] = 0.0f;
    }
  }
  const int mix = position16<D, kInt4>(gid);    // (that of gid + 8 is 8 more)
  // int4: the row of V that the lane names, and its first piece
  [[maybe_unused]] const int v_row = (lane & 7) + ((lane >> 3) & 1) * 8, v_piece = lane >> 4;
  int slot = 0;
  for (int v = v0; v < v1; v += kHop) {
    {
      const int ahead = v + (Y::kDepth - 1) * kHop;
      const int into = slot == 0 ? Y::kDepth - 1 : slot - 1;
      uint32_t b = 0;
      __syncwarp();                             // the slot has been read by all lanes
      if (ahead < v1) {
        b = start_copies(ahead, into);
        look_up(ahead + kHop);
      }
      cp_async_commit();
      bits[Y::kDepth - 1] = b;
    }
    cp_async_wait<Y::kDepth - 1>();
    __syncwarp();                               // the other lanes' copies too
    const uint32_t have = bits[0];
    const unsigned char* st = s_ring + slot * Y::kStage;
    const uint32_t* words = reinterpret_cast<const uint32_t*>(st + 2 * Y::kCodes);
    // e2m1's facts of the step
    [[maybe_unused]] float4* k_quarters = reinterpret_cast<float4*>(s_ring + Y::kDepth * Y::kStage);
    [[maybe_unused]] uint2* v_facs = reinterpret_cast<uint2*>(k_quarters + kStep);
    [[maybe_unused]] float* v_scales = reinterpret_cast<float*>(v_facs + kStep);

    // V's largest scale of the step (NaNs and infinities do not count); e2m1: a lane takes a
    // position's words apart
    uint32_t v_bits;
    if constexpr (kInt4) {
      v_bits = words[kStep + lane] & 0x7F800000u;
    } else {
      const uint32_t wk = words[lane], wv = words[kStep + lane];
      // (255, an infinity by its bits, becomes NaN; 0 is 0)
      auto scale_of = [](uint32_t bits) {
        const float x = __uint_as_float(bits & 0x7F800000u);
        return __fmaf_rn(x, 0.0f, x);
      };
      k_quarters[lane] = make_float4(scale_of(wk << 23), scale_of(wk << 15), scale_of(wk << 7),
                                     scale_of(wk >> 1));
      const uint32_t b01 = __byte_perm(wv, 0u, 0x4140), b23 = __byte_perm(wv, 0u, 0x4342);
      const uint32_t big2 = __vmaxu2(b01, b23), big = max(big2 & 0xFFFFu, big2 >> 16);
      // 2^(12 - the distance to the row's largest) as f16, 0 from 27 on
      const uint32_t less = (27u - big) & 0xFFFFu, less2 = less | (less << 16);
      v_facs[lane] = make_uint2(__viaddmax_s16x2_relu(b01, less2, 0u) << 10,
                                __viaddmax_s16x2_relu(b23, less2, 0u) << 10);
      v_bits = big << 23;
      v_scales[lane] = scale_of(v_bits);
      __syncwarp();
    }
    if (__any_sync(0xFFFFFFFFu, v_bits > top)) {
      const uint32_t now = max(
          top, __reduce_max_sync(0xFFFFFFFFu, v_bits == 0x7F800000u ? 0u : v_bits));
      const float f = now - top > (126u << 23) ? 0.0f : __uint_as_float((127u << 23) - (now - top));
      top = now;
      under = __uint_as_float((260u << 23) - top);
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if constexpr (kInt4) z_acc[nb][i] *= f;
#pragma unroll
          for (int mt = 0; mt < KCH; ++mt) acc[nb][mt][i] *= f;
        }
    }
    // scores, less the reference: s[sub][nb][i] of position sub * 16 + mix + 8 * (i >> 1), column
    // 2 tig + (i & 1)
    float s[2][NB][4];
    if constexpr (kInt4) {
      uint32_t kr[2][2][D / 32];                // the lane's piece of rows mix, mix + 8
      float ks[2][2], kz[2][2];                 // scales and zero points
#pragma unroll
      for (int sub = 0; sub < 2; ++sub)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int at = sub * 16 + mix + 8 * i;
          if constexpr (D == 128) {
            const uint4 q4 = *reinterpret_cast<const uint4*>(st + piece_at<D>(at, tig));
            kr[sub][i][0] = q4.x;
            kr[sub][i][1] = q4.y;
            kr[sub][i][2] = q4.z;
            kr[sub][i][3] = q4.w;
          } else {
            const uint2 q2 =
                *reinterpret_cast<const uint2*>(st + piece_at<D>(at, tig >> 1) + (tig & 1) * 8);
            kr[sub][i][0] = q2.x;
            kr[sub][i][1] = q2.y;
          }
          const uint32_t wd = words[at];
          ks[sub][i] = __uint_as_float(wd & 0xFFFF0000u);
          kz[sub][i] = __uint_as_float((wd & 0xFFFFu) | 0x4B000000u) - 0x1p23f;
        }
      // (the chains of products of both halves of the step side by side)
#pragma unroll
      for (int c = 0; c < D / 32; ++c) {
        uint32_t a[2][2][4];
#pragma unroll
        for (int sub = 0; sub < 2; ++sub)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const uint32_t x = kr[sub][i][c], y = x >> 8;
            a[sub][0][i] = x & 0x000F000Fu;
            a[sub][0][2 + i] = x & 0x00F000F0u;
            a[sub][1][i] = y & 0x000F000Fu;
            a[sub][1][2 + i] = y & 0x00F000F0u;
          }
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
          for (int nb = 0; nb < NB; ++nb) {
            const uint2 b = query(nb, 2 * c + k);
#pragma unroll
            for (int sub = 0; sub < 2; ++sub) {
              if (c == 0 && k == 0) mma_f16_new(s[sub][nb], a[sub][k], b.x, b.y);
              else mma_f16(s[sub][nb], a[sub][k], b.x, b.y);
            }
          }
      }
#pragma unroll
      for (int sub = 0; sub < 2; ++sub)
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int i = 0; i < 4; i += 2) {
            // (the query row's factor, then K's scale: the two multiplied first could pass float32)
            const float z = kz[sub][i >> 1];
            const float2 u = fma2(make_float2(z, z), make_float2(q_sum[nb][0], q_sum[nb][1]),
                                  make_float2(s[sub][nb][i], s[sub][nb][i + 1]));
            const float2 x = mul2(u, make_float2(row_scale[nb][0], row_scale[nb][1]));
            const float2 y = fma2(x, make_float2(ks[sub][i >> 1], ks[sub][i >> 1]),
                                  make_float2(m_neg[nb][0], m_neg[nb][1]));
            s[sub][nb][i] = y.x;
            s[sub][nb][i + 1] = y.y;
          }
    } else {
      // a quarter's products by themselves, then under its scale
#pragma unroll
      for (int sub = 0; sub < 2; ++sub) {
        float4 kq[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) kq[i] = k_quarters[sub * 16 + mix + 8 * i];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          constexpr int kPer = D / 64;          // products per quarter
          uint32_t a[kPer][4];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int at = sub * 16 + mix + 8 * i;
            if constexpr (D == 128) {
              const uint32_t x = *reinterpret_cast<const uint32_t*>(st + piece_at<D>(at, c) + tig * 4);
              a[0][i] = e2m1_f16<0>(x);
              a[0][2 + i] = e2m1_f16<1>(x);
              a[kPer - 1][i] = e2m1_f16<2>(x);
              a[kPer - 1][2 + i] = e2m1_f16<3>(x);
            } else {
              const uint32_t x = *reinterpret_cast<const uint16_t*>(st + piece_at<D>(at, c >> 1) +
                                                                    (c & 1) * 8 + tig * 2);
              a[0][i] = e2m1_f16<0>(x);
              a[0][2 + i] = e2m1_f16<1>(x);
            }
          }
#pragma unroll
          for (int nb = 0; nb < NB; ++nb) {
            float t[4];
            const uint2 b0 = query(nb, kPer * c);
            mma_f16_new(t, a[0], b0.x, b0.y);
            if constexpr (kPer == 2) {
              const uint2 b1 = query(nb, 2 * c + 1);
              mma_f16(t, a[1], b1.x, b1.y);
            }
#pragma unroll
            for (int i = 0; i < 4; i += 2) {
              const float4& k4 = kq[i >> 1];
              const float k = c == 0 ? k4.x : (c == 1 ? k4.y : (c == 2 ? k4.z : k4.w));
              const float2 x = make_float2(t[i], t[i + 1]), k2 = make_float2(k, k);
              const float2 y = c == 0 ? mul2(x, k2)
                                      : fma2(x, k2, make_float2(s[sub][nb][i], s[sub][nb][i + 1]));
              s[sub][nb][i] = y.x;
              s[sub][nb][i + 1] = y.y;
            }
          }
        }
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int i = 0; i < 4; i += 2) {
            const float2 y = fma2(make_float2(s[sub][nb][i], s[sub][nb][i + 1]),
                                  make_float2(row_scale[nb][0], row_scale[nb][1]),
                                  make_float2(m_neg[nb][0], m_neg[nb][1]));
            s[sub][nb][i] = y.x;
            s[sub][nb][i + 1] = y.y;
          }
      }
    }
    const bool whole = have == 0xFFFFFFFFu && v >= v_from && v <= v_to;
    uint32_t seen = 0xFFFFFFFFu;                // bit nb * 8 + sub * 4 + i
    if (!whole) {
      seen = 0u;
#pragma unroll
      for (int sub = 0; sub < 2; ++sub)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int at = sub * 16 + mix + 8 * (i >> 1), pp = position(v + at);
          const bool here = (have >> at) & 1u;
#pragma unroll
          for (int nb = 0; nb < NB; ++nb) {
            const int pq = pos_q[nb][i & 1];
            const bool ok = here && pp <= pq &&
                            (A.window == 0 || pp > pq - A.window || pp < A.n_sink);
            if (ok) seen |= 1u << (nb * 8 + sub * 4 + i);
            else s[sub][nb][i] = -INFINITY;
          }
        }
    }
    // the reference, where a column has none or its maximum has passed it by kLazy
    {
      float most = -INFINITY;
#pragma unroll
      for (int sub = 0; sub < 2; ++sub)
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int i = 0; i < 4; i += 2) most = max3(most, s[sub][nb][i], s[sub][nb][i + 1]);
      if (__any_sync(0xFFFFFFFFu, most > kLazy || unset != 0u)) {
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          float f[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float m = fmaxf(fmaxf(s[0][nb][e], s[0][nb][e + 2]), fmaxf(s[1][nb][e], s[1][nb][e + 2]));
            m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, 4));
            m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, 8));
            m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, 16));
            const bool none = (unset >> (nb * 2 + e)) & 1u;
            const float by = none ? (m == -INFINITY ? 0.0f : m) : (m > kLazy ? m : 0.0f);
            if (none && m != -INFINITY) unset &= ~(1u << (nb * 2 + e));
            f[e] = none ? 0.0f : ex2(-by);
            m_neg[nb][e] -= by;
            l_part[nb][e] *= f[e];
#pragma unroll
            for (int sub = 0; sub < 2; ++sub) {
              s[sub][nb][e] -= by;
              s[sub][nb][e + 2] -= by;
            }
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if constexpr (kInt4) z_acc[nb][i] *= f[i & 1];
#pragma unroll
            for (int mt = 0; mt < KCH; ++mt) acc[nb][mt][i] *= f[i & 1];
          }
        }
      }
    }
#pragma unroll
    for (int sub = 0; sub < 2; ++sub) {
      // the weights (at most 2^8), and those on V's codes: with the rows' scales, in f16 (half a step:
      // 2^-11 of a weight)
      uint32_t pf[NB][2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int at = sub * 16 + mix + 8 * i;
        const float vs = kInt4 ? __uint_as_float(words[kStep + at] & 0xFFFF0000u) : v_scales[at];
        const float vu = __fmul_rn(vs, under);
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          float2 p = make_float2(ex2(s[sub][nb][2 * i]), ex2(s[sub][nb][2 * i + 1]));
          const float2 l = add2(make_float2(l_part[nb][0], l_part[nb][1]), p);
          l_part[nb][0] = l.x;
          l_part[nb][1] = l.y;
          p = mul2(p, make_float2(vu, vu));
          if (!whole) {       // (a position out of sight keeps the weight 0 whatever its scale)
            if (!((seen >> (nb * 8 + sub * 4 + 2 * i)) & 1u)) p.x = 0.0f;
            if (!((seen >> (nb * 8 + sub * 4 + 2 * i + 1)) & 1u)) p.y = 0.0f;
          }
          pf[nb][i] = transpose8(pack_f16(p.x, p.y));
        }
      }
      if constexpr (kInt4) {                    // the zero points of rows 2 tig, 2 tig + 1, and 8 on
        uint32_t z[4] = {0u, 0u, 0u, 0u};
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint2 w2 =
              *reinterpret_cast<const uint2*>(words + kStep + sub * 16 + 2 * tig + 8 * i);
          z[2 * i] = __byte_perm(w2.x, w2.y, 0x5410) & 0x000F000Fu;
        }
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) mma_f16(z_acc[nb], z, pf[nb][0], pf[nb][1]);
        // V: matrices of eight positions by four codes, read transposed: a lane's words hold those of
        // positions 2 tig and 2 tig + 1, dims 4 gid .. 4 gid + 3 of every 32
        const uint32_t sv = smem_u32(st + Y::kCodes);
#pragma unroll
        for (int c = 0; c < D / 64; ++c) {
          uint32_t x[4];                        // dims 64 c on, positions 0 - 7 and 8 - 15; 32 dims on
          ldmatrix_x4_trans(x, sv + piece_at<D>(sub * 16 + v_row, 2 * c + v_piece));
#pragma unroll
          for (int m = 0; m < 2; ++m) {
            const uint32_t x0 = x[2 * m], x1 = x[2 * m + 1], y0 = x0 >> 8, y1 = x1 >> 8;
            const uint32_t a[2][4] = {
                {x0 & 0x000F000Fu, x0 & 0x00F000F0u, x1 & 0x000F000Fu, x1 & 0x00F000F0u},
                {y0 & 0x000F000Fu, y0 & 0x00F000F0u, y1 & 0x000F000Fu, y1 & 0x00F000F0u}};
#pragma unroll
            for (int k = 0; k < 2; ++k)
#pragma unroll
              for (int nb = 0; nb < NB; ++nb)
                mma_f16(acc[nb][4 * c + 2 * m + k], a[k], pf[nb][0], pf[nb][1]);
          }
        }
      } else {
        // V: rows 2 tig, 2 tig + 1 and 8 on; the lane's D / 8 dims of each
        uint32_t vr[4][D / 64], vf[2];          // and the factors of a pair of rows
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int at = sub * 16 + position16<D, kInt4>(2 * tig + (i & 1)) + 8 * (i >> 1);
          const unsigned char* sv = st + Y::kCodes;
          if constexpr (D == 128) {
            const uint2 q2 =
                *reinterpret_cast<const uint2*>(sv + piece_at<D>(at, gid >> 1) + (gid & 1) * 8);
            vr[i][0] = q2.x;
            vr[i][1] = q2.y;
          } else {
            vr[i][0] =
                *reinterpret_cast<const uint32_t*>(sv + piece_at<D>(at, gid >> 2) + (gid & 3) * 4);
          }
          const uint32_t f = reinterpret_cast<const uint16_t*>(v_facs + at)[gid >> 1];
          if (i & 1) vf[i >> 1] |= f << 16;
          else vf[i >> 1] = f;
        }
#pragma unroll
        for (int c = 0; c < D / 64; ++c) {
          uint32_t a[4][4];                     // the word's four products
#pragma unroll
          for (int i = 0; i < 2; ++i) {         // rows 2 tig and the next; and 8 on
            const uint32_t wa = vr[2 * i][c], wb = vr[2 * i + 1][c];
            // bytes of both rows' codes of one dim
            const uint32_t x = (wa & 0x0F0F0F0Fu) | ((wb << 4) & 0xF0F0F0F0u);
            const uint32_t y = ((wa >> 4) & 0x0F0F0F0Fu) | (wb & 0xF0F0F0F0u);
            a[0][2 * i] = mul_f16x2(e2m1_f16<0>(x), vf[i]);
            a[0][2 * i + 1] = mul_f16x2(e2m1_f16<0>(y), vf[i]);
            a[1][2 * i] = mul_f16x2(e2m1_f16<1>(x), vf[i]);
            a[1][2 * i + 1] = mul_f16x2(e2m1_f16<1>(y), vf[i]);
            a[2][2 * i] = mul_f16x2(e2m1_f16<2>(x), vf[i]);
            a[2][2 * i + 1] = mul_f16x2(e2m1_f16<2>(y), vf[i]);
            a[3][2 * i] = mul_f16x2(e2m1_f16<3>(x), vf[i]);
            a[3][2 * i + 1] = mul_f16x2(e2m1_f16<3>(y), vf[i]);
          }
#pragma unroll
          for (int k = 0; k < 4; ++k)
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) mma_f16(acc[nb][4 * c + k], a[k], pf[nb][0], pf[nb][1]);
        }
      }
    }
#pragma unroll
    for (int i = 0; i + 1 < Y::kDepth; ++i) bits[i] = bits[i + 1];
    slot = slot + 1 == Y::kDepth ? 0 : slot + 1;
  }

  // The warps' results joined; the lane's dims of acc[mt]: e2m1 gid D / 8 + 2 mt and the next one,
  // int4 32 (mt / 2) + 4 gid + 2 (mt % 2) and the next one.
  constexpr int kLd = D + 4;                       // floats per row: a quad's rows 8 banks apart
  float* s_o = reinterpret_cast<float*>(s_dyn);    // [kWarps][R][kLd], over the rings
  __shared__ float s_m[kWarps][R], s_l[kWarps][R];
  cp_async_wait<0>();
#pragma unroll
  for (int nb = 0; nb < NB; ++nb)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float l = l_part[nb][e];
#pragma unroll
      for (int o = 4; o < 32; o *= 2) l += __shfl_xor_sync(0xFFFFFFFFu, l, o);
      if (gid == 0) {
        s_m[warp][nb * 8 + 2 * tig + e] = (unset >> (nb * 2 + e)) & 1u ? -INFINITY : -m_neg[nb][e];
        s_l[warp][nb * 8 + 2 * tig + e] = l;
      }
    }
  __syncthreads();                                 // (and no ring is read any more)
  // back from the weights' power of two: 2^(top - 133), and e2m1's 2^-12
  const float back = __uint_as_float(top - (6u << 23)) * (kInt4 ? 1.0f : 0x1p-12f);
#pragma unroll
  for (int nb = 0; nb < NB; ++nb)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int rt = nb * 8 + 2 * tig + e;
      const float best = fmaxf(fmaxf(s_m[0][rt], s_m[1][rt]), fmaxf(s_m[2][rt], s_m[3][rt]));
      const float f = ex2(__fsub_rn(s_m[warp][rt], best == -INFINITY ? 0.0f : best)) * back;
      float* o = s_o + (warp * R + rt) * kLd + gid * (kInt4 ? 4 : D / 8);
#pragma unroll
      for (int mt = 0; mt < KCH; ++mt) {
        float2 y = make_float2(acc[nb][mt][e], acc[nb][mt][2 + e]);
        if constexpr (kInt4)
          y = make_float2((y.x - z_acc[nb][e]) * 0x1p24f,
                          __fmaf_rn(y.y, 0.0625f, -z_acc[nb][e]) * 0x1p24f);
        *reinterpret_cast<float2*>(o + (kInt4 ? 32 * (mt >> 1) + 2 * (mt & 1) : 2 * mt)) =
            make_float2(y.x * f, y.y * f);
      }
    }
  __syncthreads();
  // 8 dims a thread
  const int r0_end = w.tile * R, rows_end = w.len * A.G, tok0 = w.tok;
  const int64_t unit = w.unit;
  const bool direct = w.direct;
  const int lh_end = static_cast<int>(blockIdx.x % static_cast<unsigned>(A.g.H * A.nl));
  for (int i = threadIdx.x; i < R * (D / 8); i += kWarps * 32) {
    const int rt = i / (D / 8), d = (i % (D / 8)) * 8;
    const int r = r0_end + rt;
    if (r >= rows_end) continue;
    const float best = fmaxf(fmaxf(s_m[0][rt], s_m[1][rt]), fmaxf(s_m[2][rt], s_m[3][rt]));
    float l = 0.0f, y[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) y[k] = 0.0f;
#pragma unroll
    for (int wp = 0; wp < kWarps; ++wp) {
      l = __fmaf_rn(s_l[wp][rt], ex2(__fsub_rn(s_m[wp][rt], best == -INFINITY ? 0.0f : best)), l);
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
    if (direct) {
      const int tok = r / A.G;
      const int64_t row = (static_cast<int64_t>(lh_end / A.g.H) * A.tokens + tok0 + tok) * A.nq +
                          (lh_end % A.g.H) * A.G + (r - tok * A.G);
      const float inv = l == 0.0f ? 0.0f : 1.0f / l;      // a row that sees nothing: zeros
#pragma unroll
      for (int k = 0; k < 8; ++k) y[k] *= inv;
      st16(A.out + row * D + d, pack8(y));
      if (d == 0 && A.lse)
        A.lse[row] = l == 0.0f ? -INFINITY : (best + log2f(l)) * 0.69314718055994530942f;
    } else {
      float* po = A.part_o + (unit * R + rt) * D + d;
#pragma unroll
      for (int k = 0; k < 8; k += 4)
        *reinterpret_cast<float4*>(po + k) = make_float4(y[k], y[k + 1], y[k + 2], y[k + 3]);
      if (d == 0) {
        A.part_ml[(unit * R + rt) * 2] = best;
        A.part_ml[(unit * R + rt) * 2 + 1] = l;
      }
    }
  }
}

// The block's first tile: sequence x, `at` places into its tiles of `steps` steps; unit: that of its
// part of the sequence's first tile.
__device__ __forceinline__ void enter(const Cut& cut, Place& w, int x, int64_t at, int steps,
                                      int64_t unit) {
  const int64_t each = tile_places(cut.crossing, cut.share, steps);
  const int tile = static_cast<int>(at / each);
  const int64_t off = at - tile * each;
  w.x = x;
  w.tile = tile;
  w.unit = unit + (cut.crossing ? tile : 0);
  // (in the places before the tile's steps: they are lost)
  const int64_t lost = cut.crossing ? max(kEnter - off, static_cast<int64_t>(0)) : 0;
  w.left = cut.share - lost;
  w.v_begin = static_cast<int>(cut.crossing ? max(off - kEnter, static_cast<int64_t>(0)) : off * cut.share) *
              kHop;
}
// How much of its tile the block takes; it has `left` steps left.
__device__ __forceinline__ void take(Place& w, int steps) {
  w.n = static_cast<int>(
      max(min(w.left, static_cast<int64_t>(steps - w.v_begin / kHop)), static_cast<int64_t>(0)));
  w.v_end = w.v_begin + w.n * kHop;
  w.direct = w.n == steps;
}
// On to the next tile (the caller to the next sequence).
__device__ __forceinline__ void leave(int crossing, Place& w) {
  w.left = crossing ? w.left - w.n - kEnter : 0;
  w.v_begin = 0;
  ++w.unit;
  ++w.tile;
}

// The units of tile y, which begins at s and has `steps` steps (td_internal.h: Cut).
struct Parts {
  int64_t first;
  int n;
  __device__ __forceinline__ Parts(const Cut& cut, int64_t s, int steps, int64_t y) {
    if (cut.crossing) {
      const int64_t c0 = (s + kEnter) / cut.share;
      first = c0 + y;
      n = steps == 0 ? 0 : static_cast<int>((s + kEnter + steps - 1) / cut.share - c0) + 1;
    } else {
      first = s;
      n = static_cast<int>((steps + cut.share - 1) / cut.share);
    }
  }
};

}  // namespace

// Chunks.
template <int D, int kKind, int NB>
__global__ void __launch_bounds__(kWarps * 32, token4_blocks(8 * NB, D))
chunk4_rows_kernel(const __grid_constant__ ChunkArgs A, const __grid_constant__ ChunkList list,
                   const __grid_constant__ ChunkUnits units) {
  extern __shared__ __align__(128) unsigned char s_dyn[];
  __shared__ Place s_place;
  if (threadIdx.x == 0) {                    // the block's first step
    const int heads = A.g.H * A.nl;          // (the heads of one part side by side)
    const int c = blockIdx.x / heads, lh = blockIdx.x - c * heads;
    const int s = A.cut.crossing ? c * static_cast<int>(A.cut.share) : c;
    int x = 0;
    for (int hi = list.n - 1; x < hi;) {
      const int mid = (x + hi + 1) >> 1;
      if (units.base[mid] <= s) x = mid;
      else hi = mid - 1;
    }
    enter(A.cut, s_place, x, s - units.base[x], units.nsplit[x],
          static_cast<int64_t>(lh) * A.cut.units + c + (A.cut.crossing ? units.whole[x] : 0));
  }
  pdl_wait();     // (above, the kernel's own arguments only)
  while (true) {
    if (threadIdx.x == 0) {
      const int x = s_place.x;
      s_place.agent = list.agent[x];
      s_place.start = list.start[x];
      s_place.len = list.row[x + 1] - list.row[x];
      s_place.tok = list.tok[x];
      take(s_place, units.nsplit[x]);
    }
    __syncthreads();
    if (s_place.n > 0) attend<D, kKind, NB>(A, s_place, s_dyn);
    __syncthreads();
    if (threadIdx.x == 0) {                  // the next tile, of this sequence or the next one
      leave(A.cut.crossing, s_place);
      if (s_place.tile * 8 * NB >= s_place.len * A.G) {
        s_place.tile = 0;
        if (++s_place.x == list.n) s_place.left = 0;
      }
    }
    __syncthreads();
    if (s_place.left <= 0) return;
  }
}

namespace {

// Steps of 128 positions that request x's token sees; 0 where there is nothing to see, or where the
// request is not valid.
__device__ __forceinline__ int token_steps(const TokenArgs& T, int x, int* agent, int* len) {
  const int64_t most = min(static_cast<int64_t>(T.a.pool.max_lp) * T.a.pool.P,
                           static_cast<int64_t>(INT32_MAX / 2));
  const int n = T.len[x], row = T.row ? T.row[x] : x;
  *agent = row;
  *len = n;
  if (n < 0 || n > most || row < 0 || row >= T.max_rows) {
    atomicOr(T.a.err, err_bit(TD_ERR_INVALID_ARG));
    return 0;
  }
  const int lo = T.a.window ? max(0, n - T.a.window) : 0;
  const int sinks = T.a.window ? min(T.a.n_sink, lo) : 0;
  return (sinks + n - lo + kHop - 1) / kHop;
}

// Sums over the block's warps.
__device__ __forceinline__ int64_t warp_sum(int64_t v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}

}  // namespace

// One token a request. Every block takes the sum of the requests' steps, decides the cut from it as
// all the others do, and finds its first request; block 0 leaves what the join needs.
template <int D, int kKind, int NB>
__global__ void __launch_bounds__(kWarps * 32, token4_blocks(8 * NB, D))
token4_kernel(const __grid_constant__ TokenArgs T) {
  extern __shared__ __align__(128) unsigned char s_dyn[];
  constexpr int kThreads = kWarps * 32;
  __shared__ int64_t s_sum[kWarps], s_upto[kWarps];
  __shared__ Place s_place;
  const ChunkArgs& A = T.a;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int c = blockIdx.x / (A.g.H * A.nl), lh = blockIdx.x - c * (A.g.H * A.nl);
  pdl_wait();
  // a request a thread; more than the block has threads: as many rounds, its first round's is kept
  int agent, len;
  const int own = tid < T.n ? token_steps(T, tid, &agent, &len) : 0;
  const int own_agent = agent, own_len = len;
  int64_t sum = own;
  for (int x = tid + kThreads; x < T.n; x += kThreads) sum += token_steps(T, x, &agent, &len);
  sum = warp_sum(sum);
  if (lane == 0) s_sum[warp] = sum;
  if (tid == 0) s_place.x = T.n;
  __syncthreads();
  sum = ((s_sum[0] + s_sum[1]) + (s_sum[2] + s_sum[3])) * T.tiles;
  Cut cut{kShareMin, 0, 0, 0};               // (a tile a block, if none is to be joined)
  if (T.joins) cut = cut_steps(sum, static_cast<int64_t>(T.n) * T.tiles, T.target, T.units);
  const int64_t at = cut.crossing ? static_cast<int64_t>(c) * cut.share : c;
  int64_t first = 0;                         // places of the requests before these
  for (int x0 = 0; x0 < T.n; x0 += kThreads) {
    const int x = x0 + tid;
    int steps = own;
    agent = own_agent;
    len = own_len;
    if (x0 > 0) steps = x < T.n ? token_steps(T, x, &agent, &len) : 0;
    const int64_t mine = tile_places(cut.crossing, cut.share, steps) * T.tiles;
    int64_t upto = mine;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
      const int64_t v = __shfl_up_sync(0xFFFFFFFFu, upto, o);
      if (lane >= o) upto += v;
    }
    if (lane == 31) s_upto[warp] = upto;
    __syncthreads();
    int64_t base = first + upto - mine;
    for (int i = 0; i < warp; ++i) base += s_upto[i];
    if (at >= base && at < base + mine) {
      enter(cut, s_place, x, at - base, steps,
            static_cast<int64_t>(lh) * T.units + c + (cut.crossing ? static_cast<int64_t>(x) * T.tiles : 0));
      s_place.agent = agent;
      s_place.start = len - 1;
      s_place.len = 1;
      s_place.tok = x;
      take(s_place, steps);
    }
    if (blockIdx.x == 0 && x < T.n && T.joins) {
      T.spans[x].begin = base;
      T.spans[x].steps = steps;
    }
    if (steps == 0 && c == 0 && x < T.n) {   // nothing in sight: zeros
      const int64_t row = (static_cast<int64_t>(lh / A.g.H) * T.n + x) * A.nq + (lh % A.g.H) * A.G;
      for (int i = 0; i < A.G * (D / 8); ++i) st16(A.out + row * D + i * 8, make_uint4(0u, 0u, 0u, 0u));
      for (int i = 0; A.lse && i < A.G; ++i) A.lse[row + i] = -INFINITY;
    }
    first += (s_upto[0] + s_upto[1]) + (s_upto[2] + s_upto[3]);
    __syncthreads();
  }
  if (blockIdx.x == 0 && tid == 0 && T.joins) *T.cut = cut;
  if (s_place.x == T.n) return;
  const int crossing = cut.crossing;
  while (true) {
    if (s_place.n > 0) attend<D, kKind, NB>(A, s_place, s_dyn);
    __syncthreads();
    if (tid == 0) {                          // the next tile, of this request or one that sees anything
      leave(crossing, s_place);
      int steps = 0;
      if (s_place.left > 0 && s_place.tile < T.tiles) steps = token_steps(T, s_place.x, &agent, &len);
      while (s_place.left > 0 && steps == 0) {
        s_place.unit += T.tiles - s_place.tile;
        s_place.tile = 0;
        if (++s_place.x == T.n) s_place.left = 0;
        else steps = token_steps(T, s_place.x, &agent, &len);
      }
      if (s_place.left > 0) {
        s_place.agent = agent;
        s_place.start = len - 1;
        s_place.tok = s_place.x;
        take(s_place, steps);
      }
    }
    __syncthreads();
    if (s_place.left <= 0) return;
  }
}

// The parts of every (layer, token, query head) row joined, by a block of four warps, warp w taking
// parts w, w + 4, ..., or where there are few by a warp, four rows a block. A part that saw nothing has
// the maximum -infinity, and is not used.
constexpr int kJoinWarps = 4;

namespace {

template <int D, int kWarpsRow>
__device__ __forceinline__ void join(const ChunkArgs& A, int64_t u0, int ns, int R, int rt, int64_t row) {
  constexpr int N = D / 32;
  __shared__ float s_acc[kWarpsRow][kWarpsRow > 1 ? D : 1];
  __shared__ float s_l[kWarpsRow];
  const int lane = threadIdx.x & 31, warp = kWarpsRow > 1 ? threadIdx.x >> 5 : 0;
  // this warp's first parts, on their way while the maximum is found
  constexpr int kFirst = 4;
  auto load = [&](int i, float2* ml, float* q) {
    const int64_t pr = (u0 + i) * R + rt;
    *ml = *reinterpret_cast<const float2*>(A.part_ml + pr * 2);
#pragma unroll
    for (int d = 0; d < N; d += 2) {
      const float2 f = *reinterpret_cast<const float2*>(A.part_o + pr * D + lane * N + d);
      q[d] = f.x;
      q[d + 1] = f.y;
    }
  };
  float2 ml0[kFirst];
  float q0[kFirst][N];
#pragma unroll
  for (int u = 0; u < kFirst; ++u) {
    ml0[u] = make_float2(-INFINITY, 0.0f);
    if (warp + u * kWarpsRow < ns) load(warp + u * kWarpsRow, &ml0[u], q0[u]);
  }
  float mx = -INFINITY;
  bool nan = false;
  for (int i = lane; i < ns; i += 32) {
    const float2 ml = *reinterpret_cast<const float2*>(A.part_ml + ((u0 + i) * R + rt) * 2);
    mx = fmaxf(mx, ml.x);
    nan |= ml.y != ml.y;      // scores that are NaN leave the maximum and make the sum NaN
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, o));
  nan = __any_sync(0xFFFFFFFFu, nan);
  float l = 0.0f, acc[N];
#pragma unroll
  for (int d = 0; d < N; ++d) acc[d] = 0.0f;
  auto add = [&](const float2& ml, const float* q) {
    if (ml.x == -INFINITY) return;
    const float w = exp2f(ml.x - mx);
    l = __fmaf_rn(ml.y, w, l);
#pragma unroll
    for (int d = 0; d < N; ++d) acc[d] = __fmaf_rn(q[d], w, acc[d]);
  };
#pragma unroll
  for (int u = 0; u < kFirst; ++u) add(ml0[u], q0[u]);
#pragma unroll 4
  for (int i = warp + kFirst * kWarpsRow; i < ns; i += kWarpsRow) {
    float2 ml;
    float q[N];
    load(i, &ml, q);
    add(ml, q);
  }
  if constexpr (kWarpsRow > 1) {
#pragma unroll
    for (int d = 0; d < N; ++d) s_acc[warp][lane * N + d] = acc[d];
    if (lane == 0) s_l[warp] = l;
    __syncthreads();
    if (warp != 0) return;
    l = (s_l[0] + s_l[1]) + (s_l[2] + s_l[3]);
#pragma unroll
    for (int d = 0; d < N; ++d) {
      const int k = lane * N + d;
      acc[d] = (s_acc[0][k] + s_acc[1][k]) + (s_acc[2][k] + s_acc[3][k]);
    }
  }
  if (nan) l = __uint_as_float(0x7FC00000u);
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
  uint32_t* out = reinterpret_cast<uint32_t*>(A.out + row * D + lane * N);
#pragma unroll
  for (int d = 0; d < N; d += 2) out[d / 2] = pack_bf2(acc[d] * inv, acc[d + 1] * inv);
  if (lane == 0 && A.lse)
    A.lse[row] = l == 0.0f ? -INFINITY : (mx + log2f(l)) * 0.69314718055994530942f;
}

// The row that the warp joins, or helps to.
template <int kWarpsRow>
__device__ __forceinline__ int64_t join_row() {
  constexpr int kRows = kJoinWarps / kWarpsRow;
  return static_cast<int64_t>(blockIdx.x) * kRows + (kRows > 1 ? threadIdx.x >> 5 : 0);
}

}  // namespace

template <int D, int kWarpsRow>
__global__ void __launch_bounds__(kJoinWarps * 32)
chunk4_join_kernel(const __grid_constant__ ChunkArgs A, const __grid_constant__ ChunkList list,
                   const __grid_constant__ ChunkUnits units, int R) {
  const int n_tok = list.row[list.n];
  const int64_t at = join_row<kWarpsRow>();
  const int lt = static_cast<int>(at / A.nq), gq = static_cast<int>(at - static_cast<int64_t>(lt) * A.nq);
  const int li = lt / n_tok, t = lt - li * n_tok;
  if (li >= A.nl) {
    pdl_wait();
    return;
  }
  int x = 0;
  for (int hi = list.n - 1; x < hi;) {
    const int mid = (x + hi + 1) >> 1;
    if (list.row[mid] <= t) x = mid;
    else hi = mid - 1;
  }
  const int h = gq / A.G, r = (t - list.row[x]) * A.G + gq - h * A.G, tile = r / R;
  const int steps = units.nsplit[x];
  const Parts parts(A.cut, units.base[x] + tile * tile_places(A.cut.crossing, A.cut.share, steps), steps,
                    units.whole[x] + tile);
  pdl_wait();     // (above, the kernel's own arguments only)
  if (parts.n == 1) return;                  // written already
  join<D, kWarpsRow>(A, static_cast<int64_t>(li * A.g.H + h) * A.cut.units + parts.first, parts.n, R,
                     r - tile * R, (static_cast<int64_t>(li) * A.tokens + list.tok[x] + t - list.row[x]) * A.nq + gq);
}

template <int D, int kWarpsRow>
__global__ void __launch_bounds__(kJoinWarps * 32)
token4_join_kernel(const __grid_constant__ TokenArgs T, int R) {
  const ChunkArgs& A = T.a;
  const int64_t at = join_row<kWarpsRow>();
  const int lt = static_cast<int>(at / A.nq), gq = static_cast<int>(at - static_cast<int64_t>(lt) * A.nq);
  const int li = lt / T.n, x = lt - li * T.n;
  const int h = gq / A.G, g = gq - h * A.G, tile = g / R;
  pdl_wait();
  if (li >= A.nl) return;
  const Cut cut = *T.cut;
  const int64_t begin = T.spans[x].begin;
  const int steps = T.spans[x].steps;
  const Parts parts(cut, begin + tile * tile_places(cut.crossing, cut.share, steps), steps,
                    static_cast<int64_t>(x) * T.tiles + tile);
  if (parts.n <= 1) return;                  // written already
  join<D, kWarpsRow>(A, static_cast<int64_t>(li * A.g.H + h) * T.units + parts.first, parts.n, R, g - tile * R,
                     (static_cast<int64_t>(li) * T.n + x) * A.nq + gq);
}

namespace {

// Whether a row is joined by one warp or by a block, by how many parts a tile has on average (one more
// where blocks cross the tiles' ends): two drafted tokens of 64 requests, 2 to 3 parts, 81 us by warps
// and 86 by blocks, 4 tokens of 8 requests, 7 parts, 11.3 and 11.9 in a graph, one of ten requests, 11
// parts, 15.0 and 14.4.
bool few_parts(int64_t blocks, int64_t tiles) { return blocks <= 8 * tiles; }
dim3 join_grid(int64_t rows, bool few) {
  return dim3(static_cast<unsigned>(few ? (rows + kJoinWarps - 1) / kJoinWarps : rows));
}

template <typename K>
cudaError_t allow(K* kernel, int smem, bool fresh) {
  return fresh ? cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem)
               : cudaSuccess;
}

template <int D, int kKind>
cudaError_t run_rows(const ChunkArgs& a, const ChunkList& list, const ChunkUnits& units, int rows,
                     bool fresh, cudaStream_t st) {
  using Y = Ring<D, kKind>;
  static_assert(Y::kRings >= kWarps * 16 * (D + 4) * 4, "the rings' space takes the warps' results");
  const unsigned grid = static_cast<unsigned>(a.nl) * a.g.H * a.cut.blocks;
  if (grid == 0) return cudaSuccess;
  auto* kernel = rows == 8 ? chunk4_rows_kernel<D, kKind, 1> : chunk4_rows_kernel<D, kKind, 2>;
  const cudaError_t e = allow(kernel, Y::smem(rows), fresh);
  return e != cudaSuccess ? e : launch_after(kernel, grid, kWarps * 32, Y::smem(rows), st, a, list, units);
}

template <int D, int kKind>
cudaError_t run_token(const TokenArgs& t, int rows, bool fresh, cudaStream_t st) {
  using Y = Ring<D, kKind>;
  const unsigned grid = static_cast<unsigned>(t.a.nl) * t.a.g.H * t.target;
  auto* kernel = rows == 8 ? token4_kernel<D, kKind, 1> : token4_kernel<D, kKind, 2>;
  cudaError_t e = allow(kernel, Y::smem(rows), fresh);
  if (e == cudaSuccess) e = launch_after(kernel, grid, kWarps * 32, Y::smem(rows), st, t);
  if (e != cudaSuccess || !t.joins) return e;
  const int64_t out_rows = static_cast<int64_t>(t.a.nl) * t.n * t.a.nq;
  const bool few = few_parts(t.target, static_cast<int64_t>(t.n) * t.tiles);
  return launch_after(few ? token4_join_kernel<D, 1> : token4_join_kernel<D, kJoinWarps>,
                      join_grid(out_rows, few), kJoinWarps * 32, 0, st, t, rows);
}

}  // namespace

cudaError_t launch_chunk4_rows(const ChunkArgs& a, const ChunkList& list, const ChunkUnits& units,
                               CacheKind kind, int rows_per_tile, bool fresh, cudaStream_t st) {
  const bool wide = a.g.D == 128;
  if (kind == kCacheInt4)
    return wide ? run_rows<128, kCacheInt4>(a, list, units, rows_per_tile, fresh, st)
                : run_rows<64, kCacheInt4>(a, list, units, rows_per_tile, fresh, st);
  return wide ? run_rows<128, kCacheE2m1>(a, list, units, rows_per_tile, fresh, st)
              : run_rows<64, kCacheE2m1>(a, list, units, rows_per_tile, fresh, st);
}

cudaError_t launch_chunk4_join(const ChunkArgs& a, const ChunkList& list, const ChunkUnits& units,
                               int rows_per_tile, cudaStream_t st) {
  const int64_t rows = static_cast<int64_t>(a.nl) * list.row[list.n] * a.nq;
  int64_t tiles = 0;
  for (int x = 0; x < list.n; ++x)
    tiles += (static_cast<int64_t>(list.row[x + 1] - list.row[x]) * a.G + rows_per_tile - 1) / rows_per_tile;
  const bool few = few_parts(a.cut.blocks, tiles);
  const dim3 grid = join_grid(rows, few);
  if (a.g.D == 128)
    return launch_after(few ? chunk4_join_kernel<128, 1> : chunk4_join_kernel<128, kJoinWarps>, grid,
                        kJoinWarps * 32, 0, st, a, list, units, rows_per_tile);
  return launch_after(few ? chunk4_join_kernel<64, 1> : chunk4_join_kernel<64, kJoinWarps>, grid,
                      kJoinWarps * 32, 0, st, a, list, units, rows_per_tile);
}

cudaError_t launch_token4(const TokenArgs& t, CacheKind kind, int rows_per_tile, bool fresh,
                          cudaStream_t st) {
  const bool wide = t.a.g.D == 128;
  if (kind == kCacheInt4)
    return wide ? run_token<128, kCacheInt4>(t, rows_per_tile, fresh, st)
                : run_token<64, kCacheInt4>(t, rows_per_tile, fresh, st);
  return wide ? run_token<128, kCacheE2m1>(t, rows_per_tile, fresh, st)
              : run_token<64, kCacheE2m1>(t, rows_per_tile, fresh, st);
}

}  // namespace td
