// k_chunk_tc.cu - attention of a chunk of new tokens over a paged cache, for many query rows:
// tcgen05 tensor cores, accumulators in TMEM, K and V tiles brought by TMA.
//
// The mathematics is k_chunk.cu's: token u of a chunk at pos = start + u sees p <= pos (and,
// under a window, p > pos - W or p < n_sink); out = softmax(scale q K^T) V over what it sees.
// The query rows of a kv head are the pairs (token, head of the group): a CTA takes up to 256
// of them as two tiles of 128 and walks the KV tiles of 128 positions that any of them sees:
//   S_w = Q_w K^T        (128 x 128, float32 in TMEM; operands in shared memory)
//   P_w = 2^(S_w - m)    (bf16, in TMEM: over S_w at D = 128, beside it at D = 64)
//   O_w += P_w V         (float32 in TMEM; A operand from TMEM, V as stored: dims-major)
// Warps 0-3 and 4-7 run the softmax of the two tiles, a thread a row, so that no statistic
// crosses threads; one warp issues all products; the two tiles alternate, so that the tensor
// core works on one while the other is in its softmax. Per KV tile and both query tiles the
// 4 x 2^14 D multiply-adds take 2048 cycles at D = 128 and 1024 at D = 64 (4096 a cycle), the
// 2 x 2^14 exponentials 1024 (32 a cycle): the products bound D = 128, both D = 64.
//
// Measured on one GB300: two chunks of 2048 tokens after 8192, 28 query heads on 4, D = 128,
// take 350 us = 1.54 PFLOP/s (80% of what a large library product reaches), the tensor pipe
// busy for 73% of the cycles; ragged spans of 1 to 301 tokens after 6000 to 13000, 40 heads on
// 8, reach 1.31 (whatever the page size from 8 on). Under a window of 1024 at D = 64 a block has
// 11 KV tiles, the first and last of them partly masked: 314 us = 599 TFLOP/s of visible work
// (64 heads on 8, four chunks of 1500 to 4097), a quarter of it the block's start and end and
// the rest bound by the softmax's issue. e4m3 pages, four chunks of 500 to 700 after 4096 to
// 8192, 40 heads on 8, D = 128: 262 us = 1.25 PFLOP/s with the pages unfolded first; converted
// by every block for itself they took 395. Blocks that stay and take unit after unit lost 5 to
// 22% to this grid; a single query tile a block, two blocks an SM, lost 13 to 23% at D = 64 (it
// loads K and V twice).
//
// The running maximum is lazy: the reference m is set to a row's maximum and 8 more (in base 2),
// and raised, and O rescaled (in TMEM, by the softmax warps), only when the maximum passes it.
// So no weight is over 1 (V may be next to the largest float32), and a row's largest is 2^-8 or
// more, which float32 sums and bf16's relative precision do not mind. The weights are rounded to
// bf16 (at most 2^-8 relative) for the tensor cores, as the output is; their sum is taken before, in
// float32. (Split in two parts as in the streaming kernel they would cost half the products'
// time again.)
//
// bf16 pages: a tile arrives as boxes of 8 to 128 rows x 64 dims, each inside one page
// (tensor map, 128-byte swizzle), K on a ring of its own, V on another. Every V tile passes
// a patch warp before the products read it: where a tile holds positions that some row does
// not see, it clears the rows that none sees (their bytes may be anything) and watches for
// infinities and NaNs in the others: 0 * NaN would reach rows that do not see them. Such a
// value (rare) becomes a zero in the tile, and is added to its element of the rows that see it
// after their outputs are written (add_values): no other element and no other row changes.
// 8-bit pages of long chunks are unfolded before (k_expand.cu): their tiles lie together, whole,
// with zeros where nothing is seen, and come by TMA without a table or a patch; one warp
// brings the positions' scales. For shorter chunks three warps load K's codes and four V's, turn
// them into f16 and bf16 (exact) and store them as the same tiles; the queries become f16 too,
// each row with a power of two that brings it to f16's range. Either way the scale of K's row
// goes on the score's column, that of V's on the weight's; powers of two (e4m3 as
// td_quantise_append writes it) go into the conversion itself, exactly, and cost the softmax
// nothing.
//
// Every wait is bounded by the global timer; when one runs out TD_ERR_DEVICE_TIMEOUT is set
// and all roles leave their loops, wait (bounded) for what they started and free the TMEM.
#include "td_cache8.cuh"

namespace td {

namespace {

constexpr int kKv = 128;              // positions per KV tile
constexpr int kRows = 128;            // query rows per tile
constexpr int kSoftmaxWarps = 8;
constexpr int kMmaWarp = 8;
constexpr int kLoadWarp = 9;          // bf16: K by TMA; V: the next warp
constexpr int kPatchWarp = 11;
constexpr int kConvertWarp = 12;      // 8-bit: the first of four that convert V (9-11: K)
constexpr int kInfo = 8;              // KV tiles whose facts are kept
constexpr float kLazy = 8.0f;         // the reference is set by this much over the maximum (base 2)

// Kinds of the kernel: CacheKind, or 8-bit pages' unfolded copy.
constexpr int kUnfolded = 3;
__host__ __device__ constexpr bool converts(int kind) {
  return kind == kCacheInt8 || kind == kCacheE4m3;
}

template <int D, int kKind>
struct Plan {
  static constexpr bool k8 = converts(kKind);
  static constexpr int kTile = kKv * D * 2;              // bytes of a K or V tile
  static constexpr int kQ = 2 * kRows * D * 2;
  // K and V tiles in flight. One CTA an SM either way (TMEM is taken whole): D = 64 leaves
  // room for more, and must take more than half of the shared memory
  // (at D = 128 a third K tile changed nothing)
  static constexpr int kK = D == 64 ? 4 : 2;
  static constexpr int kV = D == 64 ? 4 : 2;
  // TMEM columns: two S, two O, and at D = 64 two P of their own: the next scores may then be
  // computed while the softmax still works on the last ones (at D = 128 P lies over S)
  static constexpr bool kOwnP = D == 64;
  static constexpr uint32_t kColO = 2 * kKv, kColP = 2 * kKv + 2 * D;
  static constexpr int kThreads = k8 ? 512 : 384;
  // 8-bit pages: the last KV tiles' scales; where they are converted here, four tiles' page rows
  // (a thread may write those of tile j + 2 while another still reads tile j's)
  static constexpr int kScales = kKind != kCacheBf16 ? kInfo * 2 * kKv * 4 : 0;
  static constexpr int kPageRows = k8 ? 4 * kKv * 4 : 0;
  static constexpr int kRowScales = k8 ? 2 * kRows * 4 : 0;     // and the query rows' factors
  static constexpr int kSmem = 1024 + kQ + (kK + kV) * kTile + kScales + kPageRows + kRowScales + 1024;
};

// A KV tile's facts. Bit p of `valid`: position p's page is mapped, or nobody needs it.
// `folded` (8-bit pages): the scales of word i's positions are in the converted K and V.
struct __align__(16) Info {
  uint32_t valid[4];
  uint32_t folded[4];
  __device__ __forceinline__ bool all_folded() const {
    const volatile uint32_t* v = folded;
    return (v[0] & v[1] & v[2] & v[3]) != 0;
  }
  __device__ __forceinline__ uint4 load() const {
    const volatile uint32_t* v = valid;
    return make_uint4(v[0], v[1], v[2], v[3]);
  }
};
__device__ __forceinline__ bool no_holes(const uint4& v) { return (v.x & v.y & v.z & v.w) == ~0u; }

struct Shared {
  uint64_t q_full, k_full[4], k_empty[4], v_raw[4], v_full[4], v_empty[4];
  uint64_t s_full[2], s_empty[2], p_ready[2][2], o_done[2], drain;   // p_ready: the weights' halves
  uint32_t tmem;
  int abort, bad;
  int place[4];                      // x, h, li and unit of the CTA's work
  alignas(16) int box_row[2][16];    // K's and V's loader: rows of the tile's boxes
  Info info[kInfo];
};
static_assert(sizeof(Shared) <= 1024, "the block's bookkeeping has 1 KB");

// ---- PTX
__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}

__device__ __forceinline__ void fence_async_smem() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

__device__ __forceinline__ void tma_box(uint32_t dst, const CUtensorMap* map, int x, int y,
                                        uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3}], [%4];"
      ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(smem_u32(bar))
      : "memory");
}

__device__ __forceinline__ void tc_fence_before() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tc_fence_after() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
// Waits for the warp's loads; the loaded registers go through it (or through tc_loaded after
// it), so that nothing reads them earlier.
#define TD_R8(r, i) "+r"(r[i]), "+r"(r[i + 1]), "+r"(r[i + 2]), "+r"(r[i + 3]), \
                    "+r"(r[i + 4]), "+r"(r[i + 5]), "+r"(r[i + 6]), "+r"(r[i + 7])
__device__ __forceinline__ void tc_wait_ld(uint32_t* r) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : TD_R8(r, 0), TD_R8(r, 8), TD_R8(r, 16), TD_R8(r, 24)::"memory");
}
__device__ __forceinline__ void tc_loaded(uint32_t* r) {
  asm volatile("" : TD_R8(r, 0), TD_R8(r, 8), TD_R8(r, 16), TD_R8(r, 24)::"memory");
}
__device__ __forceinline__ void tc_wait_ld16(uint32_t* r) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" : TD_R8(r, 0), TD_R8(r, 8)::"memory");
}
#undef TD_R8
__device__ __forceinline__ void tc_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ void tc_commit(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];"
               ::"r"(smem_u32(bar)) : "memory");
}

// D (TMEM) = A B (+ D): both operands in shared memory.
__device__ __forceinline__ void tc_mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                          bool add) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}"
      ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(static_cast<uint32_t>(add))
      : "memory");
}
// The same with A in TMEM.
__device__ __forceinline__ void tc_mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc,
                                          bool add) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
      ::"r"(d), "r"(a), "l"(b), "r"(idesc), "r"(static_cast<uint32_t>(add))
      : "memory");
}

// 32 columns of the warp's 32 lanes.
__device__ __forceinline__ void tc_ld32(uint32_t* r, uint32_t addr) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
        "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
        "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(addr));
}
__device__ __forceinline__ void tc_ld16(uint32_t* r, uint32_t addr) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(addr));
}
__device__ __forceinline__ void tc_st16(uint32_t addr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};"
      ::"r"(addr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]),
        "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]),
        "r"(r[14]), "r"(r[15])
      : "memory");
}

// 16 bytes of shared memory, read where it is written.
__device__ __forceinline__ int4 lds_int4(const int* p) {
  int4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(smem_u32(p))
               : "memory");
  return v;
}

// One lane of the warp, always the same. The products' warp runs as one and only issues under
// this: its addresses and descriptors stay warp-uniform, in uniform registers (issued from a
// branch of lane 0 alone, each product cost about 100 cycles of moves, against 64 of tensor
// work).
__device__ __forceinline__ bool elected() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}"
               : "=r"(p));
  return p != 0;
}

// Shared-memory operand of 64-element (128-byte) swizzled rows: `next` = bytes between
// neighbouring 64-element column blocks (read for dims-major operands only), 1024 bytes
// between groups of 8 rows.
__device__ __forceinline__ uint64_t tc_desc(uint32_t addr, uint32_t next) {
  return static_cast<uint64_t>((addr & 0x3FFFFu) >> 4) |
         (static_cast<uint64_t>(next >> 4) << 16) | (static_cast<uint64_t>(1024 >> 4) << 32) |
         (1ull << 46) | (2ull << 61);
}

// Instruction descriptor: bf16 (or f16) operands, float32 accumulators, 128 x n; b_dims: B is
// stored with its n index contiguous.
__host__ __device__ constexpr uint32_t tc_idesc(int n, bool b_dims, bool f16) {
  return (1u << 4) | (f16 ? 0u : (1u << 7) | (1u << 10)) | (static_cast<uint32_t>(b_dims) << 16) |
         (static_cast<uint32_t>(n >> 3) << 17) | (static_cast<uint32_t>(kRows >> 4) << 24);
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n\t.reg .b64 a, b, c, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
      "mov.b64 c, {%6, %7};\n\tfma.rn.f32x2 d, a, b, c;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 a, b, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
      "add.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}

__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 a, b, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
      "mul.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}

__device__ __forceinline__ uint32_t mul2_f16(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

// Waits for a phase, for at most kWaitLimitNs or until another role gave up.
__device__ __forceinline__ bool wait_or_abort(uint64_t* bar, unsigned parity, Shared* sh,
                                              uint32_t* err) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = global_ns();
  while (true) {
    if (mbar_try_wait(bar, parity)) return true;
    if (*reinterpret_cast<volatile int*>(&sh->abort)) return false;
    if (global_ns() - t0 >= kWaitLimitNs) {
      *reinterpret_cast<volatile int*>(&sh->abort) = 1;
      atomicOr(err, err_bit(TD_ERR_DEVICE_TIMEOUT));
      return false;
    }
  }
}

// Byte offset of 16-byte chunk c of row r in a tile (64-dim column blocks of 128 rows,
// 128-byte swizzle).
__device__ __forceinline__ uint32_t tile_at(int r, int c) {
  return (c >> 3) * (128 * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4);
}

// What a CTA works on.
struct Work {
  int x, h, li;                 // sequence, kv head, layer of the launch
  int unit;                     // number of its partial results; -1: none, it has all KV tiles
                                // of its rows and writes their outputs
  int r0, nrows;                // query rows r0 .. r0 + nrows - 1 of the sequence
  int start, len;
  int p_first, p_last;          // positions of the first and the last row's tokens
  int s_tiles, t_lo;            // KV tiles: 0 .. s_tiles - 1, then t_lo ..
  int i0, n;                    // the part: KV tiles i0 .. i0 + n - 1 of that list
  int window, n_sink;

  // the part's j-th tile: under a window from the middle on, then the first ones, since those
  // at the ends are masked and their V is patched, which takes a tile's time
  __device__ __forceinline__ int tile(int j) const {
    int i = j;
    if (window) {
      i += n >> 1;
      if (i >= n) i -= n;
    }
    i += i0;
    return i < s_tiles ? i : t_lo + i - s_tiles;
  }
  // every row of tokens at positions pf .. pl sees all positions of the tile
  __device__ __forceinline__ bool whole(int kt, int pf, int pl) const {
    const int t0 = kt * kKv, t1 = t0 + kKv - 1;
    return t1 <= pf && (window == 0 || t0 > pl - window || t1 < n_sink);
  }
  // some row sees a position of [a, b]
  __device__ __forceinline__ bool needed(int a, int b) const {
    return a <= p_last && (window == 0 || b > p_first - window || a < n_sink);
  }
};

__device__ __forceinline__ Work work_of(const ChunkArgs& A, const ChunkList& list,
                                        const ChunkUnits& units) {
  Work w;
  const int total = units.base[list.n];
  const int lh = blockIdx.x % (A.g.H * A.nl);
  const int c = blockIdx.x / (A.g.H * A.nl);
  w.h = lh % A.g.H;
  w.li = lh / A.g.H;
  int x = 0;
  for (int hi = list.n - 1; x < hi;) {
    const int mid = (x + hi + 1) >> 1;
    if (units.base[mid] <= c) x = mid;
    else hi = mid - 1;
  }
  w.x = x;
  const int ns = units.nsplit[x];
  w.start = list.start[x];
  w.len = list.row[x + 1] - list.row[x];
  const int rows = w.len * A.G;
  // a sequence's last tiles see most: they start first
  const int at = c - units.base[x], whole = units.whole[x];
  const int turned = at < whole ? at : whole + (at - whole) / ns;
  const int split = at < whole ? 0 : (at - whole) % ns;
  const bool direct = A.direct || at < whole;
  const int tile = (rows + A.rows_cta - 1) / A.rows_cta - 1 - turned;
  w.unit = direct ? -1 : lh * (total - A.whole_units) + (c - A.whole_units);
  w.r0 = tile * A.rows_cta;
  w.nrows = min(A.rows_cta, rows - w.r0);
  w.p_first = w.start + w.r0 / A.G;
  w.p_last = w.start + (w.r0 + w.nrows - 1) / A.G;
  w.window = A.window;
  w.n_sink = A.n_sink;
  const int lo = A.window ? max(0, w.p_first - A.window + 1) : 0;
  const int sinks = A.window ? min(A.n_sink, lo) : 0;
  w.s_tiles = (sinks + kKv - 1) / kKv;
  w.t_lo = max(lo / kKv, w.s_tiles);
  const int all = w.s_tiles + max(0, w.p_last / kKv - w.t_lo + 1);
  w.i0 = split * A.span;
  w.n = direct ? all : min(A.span, all - w.i0);
  return w;
}

// A position's page, read ahead of its use: the table's entry (kNoPage: not looked up) and the
// slot in the page.
constexpr int kNoPage = INT32_MIN;
struct PageRef {
  int page, slot;
  // page * P + slot; -1 where it was not looked up, -2 where it is unmapped
  __device__ __forceinline__ int row(const PoolDev& P) const {
    if (page == kNoPage) return -1;
    return page < 0 || page >= P.num_pages ? -2 : page * P.P + slot;
  }
};
__device__ __forceinline__ PageRef page_ref(const PoolDev& P, int agent, int pos, bool need) {
  PageRef f;
  const int lp = P.p_shift >= 0 ? (pos >> P.p_shift) : pos / P.P;
  f.slot = pos - lp * P.P;
  f.page = !need ? kNoPage : -1;
  if (need && lp < P.max_lp) f.page = __ldg(P.bt + static_cast<int64_t>(agent) * P.max_lp + lp);
  return f;
}

// Output row (or partial) addresses of query row r (within the sequence).
__device__ __forceinline__ int64_t out_row(const ChunkArgs& A, const ChunkList& list,
                                           const Work& w, int r) {
  const int tok = r / A.G;
  return (static_cast<int64_t>(w.li) * A.tokens + list.tok[w.x] + tok) * A.nq +
         w.h * A.G + (r - tok * A.G);
}

// The lowest n bits of a word (none for n <= 0, all from 32 on).
__device__ __forceinline__ uint32_t first_bits(int n) {
  return n <= 0 ? 0u : (n >= 32 ? 0xFFFFFFFFu : (1u << n) - 1u);
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// One tile's softmax for the thread's row: all 128 scores into registers, the maximum (and,
// where it grew, O rescaled), the weights written over the scores and added to the sum. The
// products may start on the first half of the weights while the second is computed: each half
// has its barrier. `seen`: the columns in sight, 4 words. `row` (kRow): the query row's factor,
// which goes on a score before K's scale does: the score of normalised queries may reach 2^31,
// and with a large scale alone it would pass float32 where the true one does not.
template <int D, bool kScaled, bool kMask, bool kRow>
__device__ __forceinline__ bool softmax_tile(uint32_t t_s, uint32_t t_o, uint32_t t_p,
                                             uint64_t* s_empty, const uint32_t* seen,
                                             float scale, float row, const float* ks, const float* vs,
                                             bool first, uint64_t* o_done, unsigned o_parity,
                                             uint64_t* p_ready, float& m_ref, float2& sum,
                                             Shared* sh, uint32_t* err) {
  uint32_t x[4][32];
#pragma unroll
  for (int c = 0; c < 4; ++c) tc_ld32(x[c], t_s + c * 32);
  tc_wait_ld(x[0]);
#pragma unroll
  for (int c = 1; c < 4; ++c) tc_loaded(x[c]);
  constexpr bool kOwnP = Plan<D, kCacheBf16>::kOwnP;
  if constexpr (kOwnP) {
    tc_fence_before();
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(s_empty);
  }
  // Masked tiles, a chunk of 32 columns at a time: in sight of every row of the warp (as an
  // unmasked tile's), of none (no work), or of some
  uint32_t none = 0, part = 0;           // bit c: chunk c
  if constexpr (kMask) {
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      if (!__any_sync(0xFFFFFFFFu, seen[c] != 0u)) none |= 1u << c;
      else if (!__all_sync(0xFFFFFFFFu, seen[c] == 0xFFFFFFFFu)) part |= 1u << c;
    }
  }
  float mx[4];
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    mx[c] = -INFINITY;
    if (kMask && (none >> c & 1u)) continue;
    [[maybe_unused]] float4 k4;
    if constexpr (kScaled) {
#pragma unroll
      for (int i = 0; i < 32; i += 2) {
        if (i % 4 == 0) k4 = *reinterpret_cast<const float4*>(ks + c * 32 + i);
        float2 v = make_float2(__uint_as_float(x[c][i]), __uint_as_float(x[c][i + 1]));
        if constexpr (kRow) v = mul2(v, make_float2(row, row));     // (a power of two: exact)
        v = mul2(v, i % 4 == 0 ? make_float2(k4.x, k4.y) : make_float2(k4.z, k4.w));
        x[c][i] = __float_as_uint(v.x);
        x[c][i + 1] = __float_as_uint(v.y);
      }
    }
    if (kMask && (part >> c & 1u)) {
#pragma unroll
      for (int i = 0; i < 32; ++i) x[c][i] = (seen[c] >> i) & 1u ? x[c][i] : 0xFF800000u;
    }
#pragma unroll
    for (int i = 0; i < 32; i += 2)
      mx[c] = max3(mx[c], __uint_as_float(x[c][i]), __uint_as_float(x[c][i + 1]));
  }
  const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
  const float m_tile = top == -INFINITY ? top : __fmul_rn(top, scale);
  if (first) {
    m_ref = m_tile + kLazy;
  } else if (__any_sync(0xFFFFFFFFu, m_tile > m_ref)) {
    // rows that did not grow keep theirs: a row's result does not depend on the others
    const bool grow = m_tile > m_ref;
    const float m_new = m_tile + kLazy;
    const float f = grow ? ex2(m_ref - m_new) : 1.0f;
    if (grow) m_ref = m_new;
    sum.x *= f;
    sum.y *= f;
    if (!__all_sync(0xFFFFFFFFu, wait_or_abort(o_done, o_parity, sh, err))) return false;
    tc_fence_after();
#pragma unroll 1
    for (int c = 0; c < D / 16; ++c) {
      uint32_t o[16];
      tc_ld16(o, t_o + c * 16);
      tc_wait_ld16(o);
#pragma unroll
      for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
      tc_st16(t_o + c * 16, o);
    }
  }
  if constexpr (kOwnP) {        // the last weights have been used
    if (!first && !__all_sync(0xFFFFFFFFu, wait_or_abort(o_done, o_parity, sh, err))) return false;
    tc_fence_after();
  }
  const float nm = m_ref == -INFINITY ? 0.0f : -m_ref;
  const float2 nm2 = make_float2(nm, nm), sc2 = make_float2(scale, scale);
  float2 sum2 = make_float2(0.0f, 0.0f);
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    uint32_t p[16];
    [[maybe_unused]] float4 v4;
    if (kMask && (none >> c & 1u)) {
#pragma unroll
      for (int i = 0; i < 16; ++i) p[i] = 0u;
    } else {
#pragma unroll
      for (int i = 0; i < 32; i += 2) {
        float2 s = make_float2(__uint_as_float(x[c][i]), __uint_as_float(x[c][i + 1]));
        s = fma2(s, sc2, nm2);
        float2 w = make_float2(ex2(s.x), ex2(s.y));
        if (c & 1) sum = add2(sum, w);
        else sum2 = add2(sum2, w);
        if constexpr (kScaled) {
          if (i % 4 == 0) v4 = *reinterpret_cast<const float4*>(vs + c * 32 + i);
          w = mul2(w, i % 4 == 0 ? make_float2(v4.x, v4.y) : make_float2(v4.z, v4.w));
          if constexpr (kMask) {      // a scale out of sight may be a NaN
            w.x = (seen[c] >> i) & 1u ? w.x : 0.0f;
            w.y = (seen[c] >> (i + 1)) & 1u ? w.y : 0.0f;
          }
        }
        p[i / 2] = pack_bf2(w.x, w.y);
      }
    }
    tc_st16(t_p + c * 16, p);
    if (c & 1) {
      tc_wait_st();
      tc_fence_before();
      __syncwarp();
      if ((threadIdx.x & 31) == 0) mbar_arrive(p_ready + (c >> 1));
    }
  }
  sum = add2(sum, sum2);
  return true;
}

// The K tiles (96 threads; f16) or V tiles (128; bf16) of a CTA, from 8-bit codes. V's threads
// also look the positions up, one each, and publish the tile's facts and scales.
template <int D, int kKind, bool kV>
__device__ __forceinline__ void convert_tiles(const ChunkArgs& A, const ChunkList& list,
                                              const Work& w, int t, unsigned char* ring,
                                              float* s_scale, int* s_rows, Shared* sh) {
  using PL = Plan<D, kKind>;
  constexpr int kVec = D / 16;                          // 16-byte vectors of codes per row
  constexpr int kThreads = kV ? 128 : 96;
  constexpr int kAll = kKv * kVec;
  // vectors are taken several a thread at a time, the next ones on their way meanwhile (K's
  // conversion is shorter, so more of it covers a load); the loop over the groups stays a loop
  // (unrolled, the two converters and the softmax together ran out of the instruction cache)
  constexpr int kMany = kV || D == 64 ? 4 : 6;
  constexpr int kGroups = (kAll + kMany * kThreads - 1) / (kMany * kThreads);
  constexpr int kSlots = kV ? PL::kV : PL::kK;
  const int lane = t & 31;
  const PoolDev& P = A.pool;
  const int64_t half = P.num_pages * P.P;
  const int64_t plane = (static_cast<int64_t>(A.layer_begin + w.li) * 2) * half;
  const uint8_t* src = reinterpret_cast<const uint8_t*>(P.base) +
                       (plane + (kV ? half : 0)) * A.g.E + w.h * D;
  uint64_t* full = kV ? sh->v_full : sh->k_full;
  uint64_t* empty = kV ? sh->v_empty : sh->k_empty;
  auto lookup = [&](int j) {
    const int pos = w.tile(min(j, w.n - 1)) * kKv + t;
    return page_ref(P, list.agent[w.x], pos, j < w.n && w.needed(pos, pos));
  };
  uint4 code[kMany];
  auto load = [&](int j, int group) {
    int row[kMany];
#pragma unroll
    for (int i = 0; i < kMany; ++i) {
      const int v = t + (group * kMany + i) * kThreads;
      row[i] = v < kAll ? s_rows[(j & 3) * kKv + v / kVec] : -1;
    }
#pragma unroll
    for (int i = 0; i < kMany; ++i) {
      code[i] = make_uint4(0u, 0u, 0u, 0u);
      if (row[i] >= 0)
        code[i] = __ldg(reinterpret_cast<const uint4*>(
            src + static_cast<int64_t>(row[i]) * A.g.E + (t % kVec) * 16));
    }
  };
  float ks = 0.0f, vs = 0.0f;
  auto load_scales = [&](int row) {
    ks = vs = 0.0f;
    if (row >= 0) {
      ks = __ldg(A.scale + (plane + row) * A.g.H + w.h);
      vs = __ldg(A.scale + (plane + half + row) * A.g.H + w.h);
    }
  };
  auto group_sync = [] { asm volatile("bar.sync 1, 224;" ::: "memory"); };
  // a scale that goes into the converted values: a power of two of at most 2^7 and, for K in
  // f16, at least 2^-15 (as td_quantise_append writes e4m3's for rows with amax from 448 * 2^-15
  // to 448 * 2^7), or that of an absent row
  auto folds = [](float s) {
    return (__float_as_uint(s) & 0x007FFFFFu) == 0 && s >= 0.0f && s <= 128.0f;
  };
  int row = -1;
  PageRef next{kNoPage, 0};
  if constexpr (kV) {
    row = lookup(0).row(P);
    s_rows[t] = row;
    next = lookup(1);
  }
  group_sync();
  load(0, 0);
  if constexpr (kV) load_scales(row);
  int slot = 0, parity = 1;
  bool ok = true;                         // after a time-out the group still meets its barriers
  for (int j = 0; j < w.n; ++j) {
    Info& info = sh->info[j % kInfo];
    float* scales = s_scale + (j % kInfo) * 2 * kKv;
    if constexpr (kV) {
      const uint32_t hole = __ballot_sync(0xFFFFFFFFu, row == -2);
      const bool fold =
          kKind == kCacheE4m3 &&
          __all_sync(0xFFFFFFFFu, folds(ks) && (ks == 0.0f || ks >= 0x1p-15f) && folds(vs));
      if (hole && lane == 0) atomicOr(A.err, err_bit(TD_ERR_UNMAPPED_PAGE));
      if (lane == 0) {
        info.valid[t >> 5] = ~hole;
        info.folded[t >> 5] = fold;
      }
      scales[t] = ks;
      scales[kKv + t] = vs;
      row = next.row(P);
      s_rows[((j + 1) & 3) * kKv + t] = row;
    }
    group_sync();
    if constexpr (kV) {
      next = lookup(j + 2);
      load_scales(row);
    }
    if (ok && j >= kSlots) ok = wait_or_abort(&empty[slot], parity, sh, A.err);
    unsigned char* tile = ring + slot * PL::kTile;
    const bool fold = kKind == kCacheE4m3 && info.all_folded();
    const int c = (t % kVec) * 2;
    // D = 128: the lanes of the second 64 dims store their halves the other way round, so that
    // eight lanes meet eight bank groups
    const bool swap = D == 128 && (c & 8);
#pragma unroll 1
    for (int group = 0; group < kGroups; ++group) {
      uint4 q[kMany];
#pragma unroll
      for (int i = 0; i < kMany; ++i) q[i] = code[i];
      if (group + 1 < kGroups) load(j, group + 1);
      else load(j + 1, 0);
#pragma unroll
      for (int i = 0; i < kMany; ++i) {
        const int v = t + (group * kMany + i) * kThreads;
        if (!ok || v >= kAll) break;
        const int r = v / kVec;
        uint4 a, b;
        if constexpr (kV) {
          uint32_t f = kE4m3Factor;
          if constexpr (kKind == kCacheE4m3) {
            const uint32_t g = __float_as_uint(scales[kKv + r] * 0x1p120f) >> 16;
            f = fold ? g | (g << 16) : f;
          }
          a = make_uint4(word_bf16<kKind, false>(q[i].x, f), word_bf16<kKind, true>(q[i].x, f),
                         word_bf16<kKind, false>(q[i].y, f), word_bf16<kKind, true>(q[i].y, f));
          b = make_uint4(word_bf16<kKind, false>(q[i].z, f), word_bf16<kKind, true>(q[i].z, f),
                         word_bf16<kKind, false>(q[i].w, f), word_bf16<kKind, true>(q[i].w, f));
        } else {
          a = make_uint4(word_f16<kKind, false>(q[i].x), word_f16<kKind, true>(q[i].x),
                         word_f16<kKind, false>(q[i].y), word_f16<kKind, true>(q[i].y));
          b = make_uint4(word_f16<kKind, false>(q[i].z), word_f16<kKind, true>(q[i].z),
                         word_f16<kKind, false>(q[i].w), word_f16<kKind, true>(q[i].w));
          if constexpr (kKind == kCacheE4m3) {
            const float g = fold ? scales[r] : 1.0f;
            const uint32_t f = pack_f16(g, g);
            a = make_uint4(mul2_f16(a.x, f), mul2_f16(a.y, f), mul2_f16(a.z, f), mul2_f16(a.w, f));
            b = make_uint4(mul2_f16(b.x, f), mul2_f16(b.y, f), mul2_f16(b.z, f), mul2_f16(b.w, f));
          }
        }
        *reinterpret_cast<uint4*>(tile + tile_at(r, swap ? c + 1 : c)) = swap ? b : a;
        *reinterpret_cast<uint4*>(tile + tile_at(r, swap ? c : c + 1)) = swap ? a : b;
      }
    }
    if (ok) {
      fence_async_smem();
      mbar_arrive(&full[slot]);
    }
    if (++slot == kSlots) {
      slot = 0;
      parity ^= 1;
    }
  }
}

// V's infinities and NaNs that some of the CTA's rows see and others do not, which the patch
// warp made zeros: added to their element of the rows that see them. A weight is positive, so
// the sum with it is that infinity or a NaN whatever the weight, and an output that is written
// or a part's sum takes the value as it is. A warp finds the positions of a tile, a lane a
// position; it takes every eighth row.
template <int D>
__device__ __noinline__ void add_values(const ChunkArgs& A, const ChunkList& list,
                                        const ChunkUnits& units, int warp) {
  constexpr int N = D / 32;
  const Work w = work_of(A, list, units);
  const int lane = threadIdx.x & 31;
  const PoolDev& P = A.pool;
  const int64_t vplane = (static_cast<int64_t>(A.layer_begin + w.li) * 2 + 1) * P.num_pages * P.P;
  const uint16_t* v = P.base + vplane * A.g.E + w.h * D;
  for (int j = 0; j < w.n; ++j) {
    for (int first = 0; first < kKv; first += 32) {
      const int mine = w.tile(j) * kKv + first + lane;
      const bool all = mine <= w.p_first &&
                       (w.window == 0 || mine > w.p_last - w.window || mine < w.n_sink);
      const int row = page_ref(P, list.agent[w.x], mine, w.needed(mine, mine) && !all).row(P);
      bool bad = false;
      for (int c = 0; row >= 0 && c < D; c += 8) {
        const uint4 q = ldg16(v + static_cast<int64_t>(row) * A.g.E + c);
        bad = bad || nonfinite2(q.x) || nonfinite2(q.y) || nonfinite2(q.z) || nonfinite2(q.w);
      }
      for (uint32_t left = __ballot_sync(0xFFFFFFFFu, bad); left; left &= left - 1) {
        const int at = __ffs(left) - 1, p = w.tile(j) * kKv + first + at;
        const uint16_t* x = v + static_cast<int64_t>(__shfl_sync(0xFFFFFFFFu, row, at)) * A.g.E;
        for (int rr = warp; rr < w.nrows; rr += kSoftmaxWarps) {
          const int pos = w.start + (w.r0 + rr) / A.G;
          if (p > pos || (w.window && p <= pos - w.window && p >= w.n_sink)) continue;
          for (int d = lane * N; d < lane * N + N; ++d) {
            if ((x[d] & 0x7F80u) != 0x7F80u) continue;
            const float val = __uint_as_float(static_cast<uint32_t>(x[d]) << 16);
            if (w.unit < 0) {
              uint16_t* o = A.out + out_row(A, list, w, w.r0 + rr) * D + d;
              const float sum = __uint_as_float(static_cast<uint32_t>(*o) << 16) + val;
              *o = static_cast<uint16_t>(pack_bf2(sum, 0.0f));
            } else {
              A.part_o[(static_cast<int64_t>(w.unit) * A.rows_cta + rr) * D + d] += val;
            }
          }
        }
      }
    }
  }
}

}  // namespace

template <int D, int kKind>
__global__ void __launch_bounds__(Plan<D, kKind>::kThreads, 1)
chunk_tc_kernel(const __grid_constant__ ChunkArgs A, const __grid_constant__ ChunkList list,
                const __grid_constant__ ChunkUnits units, const __grid_constant__ DenseTiles dense,
                const __grid_constant__ CUtensorMap map) {
  using PL = Plan<D, kKind>;
  constexpr bool k8 = PL::k8, kScaled = kKind != kCacheBf16;
  extern __shared__ unsigned char s_dyn[];
  const Work w = work_of(A, list, units);
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xFFFFFFFFu, tid >> 5, 0);    // known to be the warp's
  if (w.n <= 0) {           // a part past the visible positions of its rows: empty
    pdl_wait();
    float* ml = A.part_ml + static_cast<int64_t>(w.unit) * A.rows_cta * 2;
    for (int rr = tid; rr < w.nrows; rr += PL::kThreads) {
      ml[rr * 2] = -INFINITY;
      ml[rr * 2 + 1] = 0.0f;
    }
    return;
  }
  unsigned char* base = s_dyn + ((1024 - (smem_u32(s_dyn) & 1023)) & 1023);
  unsigned char* s_q = base;
  unsigned char* s_k = base + PL::kQ;
  unsigned char* s_v = s_k + PL::kK * PL::kTile;
  float* s_scale = reinterpret_cast<float*>(s_v + PL::kV * PL::kTile);
  int* s_rows = reinterpret_cast<int*>(reinterpret_cast<unsigned char*>(s_scale) + PL::kScales);
  float* s_row_scale =
      reinterpret_cast<float*>(reinterpret_cast<unsigned char*>(s_rows) + PL::kPageRows);
  Shared* sh = reinterpret_cast<Shared*>(reinterpret_cast<unsigned char*>(s_row_scale) +
                                         PL::kRowScales);
  const bool two = w.nrows > kRows;      // both query tiles in use

  if (tid == 0) {
    mbar_init(&sh->q_full, two ? 256 : 128);
    for (int i = 0; i < PL::kK; ++i) {
      mbar_init(&sh->k_full[i], k8 ? 96 : 1);
      mbar_init(&sh->k_empty[i], 1);
    }
    for (int i = 0; i < PL::kV; ++i) {
      mbar_init(&sh->v_raw[i], 1);
      mbar_init(&sh->v_full[i], k8 ? 128 : 1);
      mbar_init(&sh->v_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh->s_full[i], 1);
      mbar_init(&sh->s_empty[i], 4);
      mbar_init(&sh->p_ready[i][0], 4);
      mbar_init(&sh->p_ready[i][1], 4);
      mbar_init(&sh->o_done[i], 1);
    }
    mbar_init(&sh->drain, 1);
    sh->abort = 0;
    sh->bad = 0;
    sh->place[0] = w.x;
    sh->place[1] = w.h;
    sh->place[2] = w.li;
    sh->place[3] = w.unit;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  pdl_wait();               // (above, the kernel's own arguments and the block's shared memory)
  // The TMEM only after the wait: a block that held it while it waited for the previous kernel
  // would keep that kernel's own blocks from theirs, if they allocate after they let this one
  // start, and neither would end.
  if (warp == kMmaWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;"
                 ::"r"(smem_u32(&sh->tmem)) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    tc_fence_before();
  }
  __syncthreads();
  pdl_trigger();
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(&sh->tmem);

  // registers: from the warps that only start copies and products to the softmax (the shares
  // add up to the launch's: 256 x 200 + 128 x 104 = 384 x 168, and for 8-bit pages
  // 256 x 168 + 256 x 88 = 512 x 128)
  if constexpr (!k8) {
    if (warp < kSoftmaxWarps) asm volatile("setmaxnreg.inc.sync.aligned.u32 200;");
    else asm volatile("setmaxnreg.dec.sync.aligned.u32 104;");
  } else {
    if (warp < kSoftmaxWarps) asm volatile("setmaxnreg.inc.sync.aligned.u32 168;");
    else asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
  }
  if (warp < kSoftmaxWarps) {
    // ------------------------------------------------------------------ softmax
    const int wg = warp >> 2;
    const int t = tid & 127;               // the row within the query tile, and the TMEM lane
    if (wg == 0 || two) {
      {  // the query tile, rows past the last one zero; a negative scale turns the query's sign
        const uint32_t flip = A.scale_log2 < 0.0f ? 0x80008000u : 0u;
        unsigned char* dst = s_q + wg * (PL::kQ / 2);
        constexpr int kVec = D / 8, kStep = kRows / kVec;     // a thread's rows are kStep apart
        const int c = t % kVec;
        int r = w.r0 + wg * kRows + t / kVec;
        int tok = r / A.G, g = r - tok * A.G;
        const int dt = kStep / A.G, dg = kStep - dt * A.G;
        const uint16_t* src =
            A.q + ((static_cast<int64_t>(w.li) * A.tokens + list.tok[w.x]) * A.nq + w.h * A.G) * D +
            c * 8;
        uint4 val[kVec];
#pragma unroll
        for (int i = 0; i < kVec; ++i) {
          val[i] = r < w.r0 + w.nrows
                       ? ldg16(src + (static_cast<int64_t>(tok) * A.nq + g) * D)
                       : make_uint4(0u, 0u, 0u, 0u);
          r += kStep;
          tok += dt;
          g += dg;
          if (g >= A.G) {
            g -= A.G;
            ++tok;
          }
        }
#pragma unroll
        for (int i = 0; i < kVec; ++i) {
          if constexpr (k8) {      // f16 (K is), the row brought to its range: kVec lanes a row
            uint32_t m = __vmaxu2(__vmaxu2(val[i].x & 0x7FFF7FFFu, val[i].y & 0x7FFF7FFFu),
                                  __vmaxu2(val[i].z & 0x7FFF7FFFu, val[i].w & 0x7FFF7FFFu));
#pragma unroll
            for (int o = kVec / 2; o > 0; o >>= 1)
              m = __vmaxu2(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
            float inverse, f[8];
            const float mul = f16_scale(max(m & 0xFFFFu, m >> 16), &inverse);
            unpack8(val[i], f);
            val[i] = make_uint4(pack_f16(f[0] * mul, f[1] * mul), pack_f16(f[2] * mul, f[3] * mul),
                                pack_f16(f[4] * mul, f[5] * mul), pack_f16(f[6] * mul, f[7] * mul));
            if (c == 0) s_row_scale[wg * kRows + t / kVec + i * kStep] = inverse;
          }
          *reinterpret_cast<uint4*>(dst + tile_at(t / kVec + i * kStep, c)) =
              make_uint4(val[i].x ^ flip, val[i].y ^ flip, val[i].z ^ flip, val[i].w ^ flip);
        }
        fence_async_smem();
        mbar_arrive(&sh->q_full);
      }
      const int rr = wg * kRows + t;
      const bool live = rr < w.nrows;
      const int pos = live ? w.start + (w.r0 + rr) / A.G : -1;
      // positions of the query tile's first and last row
      const int pf = w.start + (w.r0 + wg * kRows) / A.G;
      const int pl = w.start + (w.r0 + min(wg * kRows + kRows, w.nrows) - 1) / A.G;
      const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
      const uint32_t t_s = tmem + lanes + wg * kKv, t_o = tmem + lanes + PL::kColO + wg * D;
      const uint32_t t_p = PL::kOwnP ? tmem + lanes + PL::kColP + wg * (kKv / 2) : t_s;
      uint64_t* s_empty = &sh->s_empty[wg];
      // (never 0 below, which would turn the -infinity of a masked score into a NaN: the least
      // float32, under which no score is more than 2^-21)
      const float scale = fmaxf(fabsf(A.scale_log2), 0x1p-149f);
      bool ok = true;
      if constexpr (k8)            // (the queries' factors are the other threads')
        ok = __all_sync(0xFFFFFFFFu, wait_or_abort(&sh->q_full, 0, sh, A.err));
      const float row = k8 ? s_row_scale[rr] : 1.0f;
      float m_ref = -INFINITY;
      float2 sum = make_float2(0.0f, 0.0f);
      for (int j = 0; ok && j < w.n; ++j) {
        // (the tensor memory's loads and stores are the whole warp's: it goes on or not as one)
        ok = __all_sync(0xFFFFFFFFu, wait_or_abort(&sh->s_full[wg], j & 1, sh, A.err));
        if (!ok) break;
        tc_fence_after();
        const int kt = w.tile(j);
        const uint4 valid = sh->info[j % kInfo].load();
        const float* ks = s_scale + (j % kInfo) * 2 * kKv;
        const bool scaled = kScaled && !sh->info[j % kInfo].all_folded();
        // the query row's factor, by itself or (no scales on the scores) with the softmax's
        const float once = k8 ? fmaxf(scale * row, 0x1p-149f) : scale;
        if (!w.whole(kt, pf, pl) || !no_holes(valid)) {
          const uint32_t in[4] = {valid.x, valid.y, valid.z, valid.w};
          uint32_t seen[4];
          const int hi = pos - kt * kKv, sk = w.n_sink - kt * kKv;
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            uint32_t b = first_bits(hi + 1 - c * 32);
            if (w.window) b &= ~first_bits(hi - w.window + 1 - c * 32) | first_bits(sk - c * 32);
            seen[c] = b & in[c];
          }
          ok = scaled ? softmax_tile<D, kScaled, true, k8>(
                            t_s, t_o, t_p, s_empty, seen, scale, row, ks, ks + kKv, j == 0,
                            &sh->o_done[wg], (j - 1) & 1, sh->p_ready[wg], m_ref, sum, sh, A.err)
                      : softmax_tile<D, false, true, false>(
                            t_s, t_o, t_p, s_empty, seen, once, row, ks, ks + kKv, j == 0,
                            &sh->o_done[wg], (j - 1) & 1, sh->p_ready[wg], m_ref, sum, sh, A.err);
        } else {
          ok = scaled ? softmax_tile<D, kScaled, false, k8>(
                            t_s, t_o, t_p, s_empty, nullptr, scale, row, ks, ks + kKv, j == 0,
                            &sh->o_done[wg], (j - 1) & 1, sh->p_ready[wg], m_ref, sum, sh, A.err)
                      : softmax_tile<D, false, false, false>(
                            t_s, t_o, t_p, s_empty, nullptr, once, row, ks, ks + kKv, j == 0,
                            &sh->o_done[wg], (j - 1) & 1, sh->p_ready[wg], m_ref, sum, sh, A.err);
        }
        if (!ok) break;
      }
      if (ok)
        ok = __all_sync(0xFFFFFFFFu, wait_or_abort(&sh->o_done[wg], (w.n - 1) & 1, sh, A.err));
      if (ok) {
        tc_fence_after();
        const float l = sum.x + sum.y;
        // (read again here: kept in registers over the loop they were spilled inside it)
        Work e = w;
        const volatile int* place = sh->place;
        e.x = place[0];
        e.h = place[1];
        e.li = place[2];
        e.unit = place[3];
        if (e.unit < 0) {
          const int64_t row = live ? out_row(A, list, e, e.r0 + rr) : -1;
          const float inv = l == 0.0f ? 0.0f : 1.0f / l;      // a row that sees nothing: zeros
          // through the query tile's place (its products have ended), so that a warp writes
          // whole rows: lane by lane a row's 16-byte pieces took 3.8 us at D = 128
          unsigned char* mine = s_q + wg * (PL::kQ / 2);
#pragma unroll
          for (int c = 0; c < D / 32; ++c) {
            uint32_t x[32];
            tc_ld32(x, t_o + c * 32);
            tc_wait_ld(x);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              float y[8];
#pragma unroll
              for (int e = 0; e < 8; ++e) y[e] = __uint_as_float(x[i * 8 + e]) * inv;
              *reinterpret_cast<uint4*>(mine + tile_at(t, c * 4 + i)) = pack8(y);
            }
          }
          __syncwarp();
          constexpr int kVec = D / 8, kPer = 32 / kVec;       // rows a step
#pragma unroll 4
          for (int i = 0; i < kVec; ++i) {
            const int from = i * kPer + lane / kVec;
            const int64_t to = __shfl_sync(0xFFFFFFFFu, row, from);
            if (to >= 0)
              st16(A.out + to * D + (lane % kVec) * 8,
                   *reinterpret_cast<const uint4*>(mine + tile_at((warp & 3) * 32 + from, lane % kVec)));
          }
          if (live && A.lse)
            A.lse[row] = l == 0.0f ? -INFINITY : (m_ref + log2f(l)) * 0.69314718055994530942f;
        } else {
          const int64_t pr = static_cast<int64_t>(e.unit) * A.rows_cta + rr;
#pragma unroll
          for (int c = 0; c < D / 32; ++c) {
            uint32_t x[32];
            tc_ld32(x, t_o + c * 32);
            tc_wait_ld(x);
            if (live) {
#pragma unroll
              for (int i = 0; i < 8; ++i)
                *reinterpret_cast<uint4*>(A.part_o + pr * D + c * 32 + i * 4) =
                    make_uint4(x[i * 4], x[i * 4 + 1], x[i * 4 + 2], x[i * 4 + 3]);
            }
          }
          if (live) {
            A.part_ml[pr * 2] = m_ref;
            A.part_ml[pr * 2 + 1] = l;
          }
        }
        tc_fence_before();
      }
    }
  } else if (warp == kMmaWarp) {
    // ---------------------------------------------------------------- the products
    constexpr uint32_t id_s = tc_idesc(kKv, false, k8), id_o = tc_idesc(D, true, false);
    const uint64_t q_desc = tc_desc(smem_u32(s_q), 16), k_desc = tc_desc(smem_u32(s_k), 16);
    const uint64_t v_desc = tc_desc(smem_u32(s_v), 128 * 128);
    // (a descriptor counts addresses in 16 bytes)
    auto scores = [&](int wg, int slot, bool last) {
      if (elected()) {
        const uint64_t a = q_desc + wg * (PL::kQ / 2 / 16), b = k_desc + slot * (PL::kTile / 16);
#pragma unroll
        for (int kc = 0; kc < D / 16; ++kc) {
          const uint32_t off = ((kc >> 2) * (128 * 128) + (kc & 3) * 32) / 16;
          tc_mma_ss(tmem + wg * kKv, a + off, b + off, id_s, kc > 0);
        }
        tc_commit(&sh->s_full[wg]);
        if (last) tc_commit(&sh->k_empty[slot]);
      }
      __syncwarp();
    };
    const int last = two ? 1 : 0;
    auto keys = [&](int slot, int parity) {       // a K tile, and its scales
      return wait_or_abort(&sh->k_full[slot], parity, sh, A.err) &&
             (kKind != kUnfolded || wait_or_abort(&sh->v_raw[slot], parity, sh, A.err));
    };
    bool ok = wait_or_abort(&sh->q_full, 0, sh, A.err) && keys(0, 0);
    ok = __all_sync(0xFFFFFFFFu, ok);
    if (ok) {
      tc_fence_after();
      scores(0, 0, !two);
      if (two) scores(1, 0, true);
    }
    int ks = 0, k_par = 0, vs = 0, v_par = 0;     // slots and the parities of their phases
    for (int j = 0; ok && j < w.n; ++j) {
      if (++ks == PL::kK) {
        ks = 0;
        k_par ^= 1;
      }
      // the next scores of a query tile: once its S is free
      auto next_scores = [&](int wg) {
        if (wg == 0) ok = keys(ks, k_par);
        if constexpr (PL::kOwnP) ok = ok && wait_or_abort(&sh->s_empty[wg], j & 1, sh, A.err);
        ok = __all_sync(0xFFFFFFFFu, ok);
        if (!ok) return;
        tc_fence_after();
        scores(wg, ks, wg == last);
      };
      if constexpr (PL::kOwnP) {
        for (int wg = 0; ok && j + 1 < w.n && wg <= last; ++wg) next_scores(wg);
      }
      for (int wg = 0; ok && wg <= last; ++wg) {
        if (wg == 0) ok = wait_or_abort(&sh->v_full[vs], v_par, sh, A.err);
        const uint32_t t_p = PL::kOwnP ? tmem + PL::kColP + wg * (kKv / 2) : tmem + wg * kKv;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          ok = ok && wait_or_abort(&sh->p_ready[wg][half], j & 1, sh, A.err);
          ok = __all_sync(0xFFFFFFFFu, ok);
          if (!ok) break;
          tc_fence_after();
          if (elected()) {
            const uint64_t b = v_desc + vs * (PL::kTile / 16);
#pragma unroll
            for (int kc = half * 4; kc < half * 4 + 4; ++kc)
              tc_mma_ts(tmem + PL::kColO + wg * D, t_p + kc * 8, b + kc * (2048 / 16), id_o,
                        j > 0 || kc > 0);
            if (half == 1) {
              tc_commit(&sh->o_done[wg]);
              if (wg == last) tc_commit(&sh->v_empty[vs]);
            }
          }
          __syncwarp();
        }
        if constexpr (!PL::kOwnP) {
          if (ok && j + 1 < w.n) next_scores(wg);
        }
      }
      if (++vs == PL::kV) {
        vs = 0;
        v_par ^= 1;
      }
    }
    // whatever was started has ended before the TMEM goes
    if (elected()) tc_commit(&sh->drain);
    __syncwarp();
    mbar_wait_bounded(&sh->drain, 0);
  } else if constexpr (kKind == kUnfolded) {
    const DenseSpan span = dense_span(w.start, w.len, w.window, w.n_sink);
    const int first = dense.base[w.x];
    if (warp < kPatchWarp) {
      // --------------------------- K (first warp) or V (second) by TMA, tiles lie together
      const bool is_v = warp != kLoadWarp;
      const int plane = (2 * w.li + is_v) * A.dense_rows;
      const int slots = is_v ? PL::kV : PL::kK;
      const uint32_t ring = smem_u32(is_v ? s_v : s_k);
      uint64_t* full = is_v ? sh->v_full : sh->k_full;
      uint64_t* empty = is_v ? sh->v_empty : sh->k_empty;
      int slot = 0, parity = 1, n = 0;                    // n: tiles started
      for (; n < w.n; ++n) {
        if (n >= slots &&
            !__all_sync(0xFFFFFFFFu, wait_or_abort(&empty[slot], parity, sh, A.err)))
          break;
        const int row = plane + (first + span.index(w.tile(n))) * kKv;
        if (elected()) {
          mbar_arrive_expect_tx(&full[slot], PL::kTile + A.tx_pad);
#pragma unroll
          for (int half = 0; half < D / 64; ++half)
            tma_box(ring + slot * PL::kTile + half * (128 * 128), &map, w.h * D + half * 64, row,
                    &full[slot]);
        }
        __syncwarp();
        if (++slot == slots) {
          slot = 0;
          parity ^= 1;
        }
      }
      // the copies that were started land before the block goes, time-out or not
      for (int i = max(0, n - slots); i < n; ++i)
        mbar_wait_bounded(&full[i % slots], (i / slots) & 1);
    } else {
      // ---------- the tiles' scales and what they tell, beside K's tiles (in V's first barrier,
      // which this kind has no other use for)
      static_assert(PL::kK <= PL::kV, "a barrier for every K tile");
      const float* src = A.dense_scale +
                         (static_cast<int64_t>(w.li) * 2 * A.g.H + w.h) * A.dense_rows;
      const int64_t v_off = static_cast<int64_t>(A.g.H) * A.dense_rows;
      auto load = [&](int j, uint4* k, uint4* v) {
        const float* at = src + (first + span.index(w.tile(min(j, w.n - 1)))) * kKv + lane * 4;
        *k = __ldg(reinterpret_cast<const uint4*>(at));
        *v = __ldg(reinterpret_cast<const uint4*>(at + v_off));
      };
      uint4 nk, nv;
      load(0, &nk, &nv);
      int slot = 0, parity = 1;
      for (int j = 0; j < w.n; ++j) {
        const uint4 k = nk, v = nv;
        load(j + 1, &nk, &nv);
        if (j >= PL::kK &&
            !__all_sync(0xFFFFFFFFu, wait_or_abort(&sh->k_empty[slot], parity, sh, A.err)))
          break;
        float* to = s_scale + (j % kInfo) * 2 * kKv + lane * 4;
        *reinterpret_cast<uint4*>(to) = k;
        *reinterpret_cast<uint4*>(to + kKv) = v;
        constexpr uint32_t kOne = 0x3F800000u;
        const uint32_t holes = (k.x == kHole) | (k.y == kHole) << 1 | (k.z == kHole) << 2 |
                               (k.w == kHole) << 3;
        const bool ones = k.x == kOne && k.y == kOne && k.z == kOne && k.w == kOne &&
                          v.x == kOne && v.y == kOne && v.z == kOne && v.w == kOne;
        uint32_t word = holes << (4 * (lane & 7));        // eight lanes make a word
#pragma unroll
        for (int o = 1; o < 8; o *= 2) word |= __shfl_xor_sync(0xFFFFFFFFu, word, o);
        const bool all = __all_sync(0xFFFFFFFFu, ones);
        if ((lane & 7) == 0) {
          sh->info[j % kInfo].valid[lane >> 3] = ~word;
          sh->info[j % kInfo].folded[lane >> 3] = all;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh->v_raw[slot]);
        if (++slot == PL::kK) {
          slot = 0;
          parity ^= 1;
        }
      }
    }
  } else if constexpr (kKind == kCacheBf16) {
    if (warp < kPatchWarp) {
      // ------------------------------------- K (first warp) or V (second) by TMA
      const bool is_v = warp != kLoadWarp;
      const PoolDev& P = A.pool;
      const int box = A.box_rows, per = kKv / box;        // boxes per 64 dims
      const int vplane = static_cast<int>(P.num_pages * P.P);
      const int plane = 2 * w.li * vplane + (is_v ? vplane : 0);
      const int slots = is_v ? PL::kV : PL::kK;
      const uint32_t ring = smem_u32(is_v ? s_v : s_k);
      uint64_t* full = is_v ? sh->v_raw : sh->k_full;
      uint64_t* empty = is_v ? sh->v_empty : sh->k_empty;
      // lane b < per looks up box b of tile j
      auto lookup = [&](int j) {
        const int pos = w.tile(min(j, w.n - 1)) * kKv + lane * box;
        return page_ref(P, list.agent[w.x], pos,
                        j < w.n && lane < per && w.needed(pos, pos + box - 1));
      };
      int slot = 0, parity = 1, n = 0;                    // n: tiles started
      PageRef next = lookup(0);
      for (; n < w.n; ++n) {
        const int row = next.row(P);
        next = lookup(n + 1);
        const uint32_t holes = __ballot_sync(0xFFFFFFFFu, row == -2);
        const uint32_t bytes = __popc(__ballot_sync(0xFFFFFFFFu, row >= 0)) * box * (D * 2u);
        if (holes && lane == 0) atomicOr(A.err, err_bit(TD_ERR_UNMAPPED_PAGE));
        if (n >= slots &&
            !__all_sync(0xFFFFFFFFu, wait_or_abort(&empty[slot], parity, sh, A.err)))
          break;
        // (both warps write a tile's facts, the same ones: each before its own barrier)
        if (lane < 4) {
          uint32_t v = 0xFFFFFFFFu;
          if (holes)
            for (int i = 0; i < 32; ++i)
              if ((holes >> ((lane * 32 + i) / box)) & 1u) v &= ~(1u << i);
          sh->info[n % kInfo].valid[lane] = v;
        }
        int* rows = sh->box_row[is_v];
        if (lane < 16) rows[lane] = row < 0 ? row : plane + row;
        __syncwarp();
        if (elected()) {
          mbar_arrive_expect_tx(&full[slot], bytes + A.tx_pad);
          const uint32_t dst = ring + slot * PL::kTile;
          // (rows by fours: one by one their latency held back pages of 8 and 24 tokens, spans
          // 736 -> 810 us; all 16 in registers made the kernel spill)
          int4 four;
#pragma unroll
          for (int b = 0; b < 16; ++b) {
            if (b % 4 == 0) four = lds_int4(rows + b);
            const int r = b % 4 == 0 ? four.x : b % 4 == 1 ? four.y : b % 4 == 2 ? four.z : four.w;
            if (b >= per || r < 0) continue;
#pragma unroll
            for (int half = 0; half < D / 64; ++half)
              tma_box(dst + half * (128 * 128) + b * box * 128, &map, w.h * D + half * 64, r,
                      &full[slot]);
          }
        }
        __syncwarp();
        if (++slot == slots) {
          slot = 0;
          parity ^= 1;
        }
      }
      // the copies that were started land before the block goes, time-out or not
      for (int i = max(0, n - slots); i < n; ++i)
        mbar_wait_bounded(&full[i % slots], (i / slots) & 1);
    } else {
      // ----------------------------------------------- V tiles patched where they must be
      int slot = 0, parity = 0;
      for (int j = 0; j < w.n; ++j) {
        const int t0 = w.tile(j) * kKv;
        if (!__all_sync(0xFFFFFFFFu, wait_or_abort(&sh->v_raw[slot], parity, sh, A.err))) break;
        const uint4 in = sh->info[j % kInfo].load();
        if (!w.whole(w.tile(j), w.p_first, w.p_last) || !no_holes(in)) {
          unsigned char* tile = s_v + slot * PL::kTile;
          bool bad = false;
          // a row a lane at a time: rows in every query row's sight stay, rows in nobody's
          // (or of no page) are cleared, the others are looked through
          for (int r = lane; r < kKv; r += 32) {
            const int p = t0 + r;
            const uint32_t word = r < 64 ? (r < 32 ? in.x : in.y) : (r < 96 ? in.z : in.w);
            const bool have = w.needed(p, p) && ((word >> lane) & 1u);
            if (have && p <= w.p_first &&
                (w.window == 0 || p > w.p_last - w.window || p < w.n_sink))
              continue;
            uint32_t top = 0;     // the largest magnitudes of the halves, as bits
#pragma unroll
            for (int c = 0; c < D / 8; ++c) {
              uint4* at = reinterpret_cast<uint4*>(tile + tile_at(r, c));
              if (have) {
                const uint4 v = *at;
                top = __vmaxu2(__vmaxu2(top, __vmaxu2(v.x & 0x7FFF7FFFu, v.y & 0x7FFF7FFFu)),
                               __vmaxu2(v.z & 0x7FFF7FFFu, v.w & 0x7FFF7FFFu));
              } else {
                *at = make_uint4(0u, 0u, 0u, 0u);
              }
            }
            if ((top & 0xFFFFu) < 0x7F80u && (top >> 16) < 0x7F80u) continue;
            bad = true;           // (add_values reads the pages: the tile's value may go)
            uint16_t* at = reinterpret_cast<uint16_t*>(tile);
#pragma unroll 1
            for (int d = 0; d < D; ++d) {
              uint16_t* e = at + tile_at(r, d >> 3) / 2 + (d & 7);
              if ((*e & 0x7F80u) == 0x7F80u) *e = 0;
            }
          }
          if (bad) *reinterpret_cast<volatile int*>(&sh->bad) = 1;
          fence_async_smem();
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh->v_full[slot]);
        if (++slot == PL::kV) {
          slot = 0;
          parity ^= 1;
        }
      }
    }
  } else {
    // ------------------------- K and V from 8-bit codes: warps 12-15 make V, 9-11 K
    if (warp < kConvertWarp)
      convert_tiles<D, kKind, false>(A, list, w, tid - kLoadWarp * 32, s_k, s_scale, s_rows, sh);
    else
      convert_tiles<D, kKind, true>(A, list, w, tid - kConvertWarp * 32, s_v, s_scale, s_rows, sh);
  }

  __syncthreads();
  if constexpr (kKind == kCacheBf16) {
    if (sh->bad && !sh->abort && warp < kSoftmaxWarps) add_values<D>(A, list, units, warp);
  }
  if (warp == kMmaWarp) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
  }
}

template <int D, int kKind>
static cudaError_t run_tc(const ChunkArgs& a, const ChunkList& list, const ChunkUnits& units,
                          const DenseTiles& dense, const CUtensorMap& map, bool fresh,
                          cudaStream_t st) {
  using PL = Plan<D, kKind>;
  const unsigned grid = static_cast<unsigned>(units.base[list.n]) * a.g.H * a.nl;
  if (fresh) {
    const cudaError_t e = cudaFuncSetAttribute(
        chunk_tc_kernel<D, kKind>, cudaFuncAttributeMaxDynamicSharedMemorySize, PL::kSmem);
    if (e != cudaSuccess) return e;
  }
  return launch_after(chunk_tc_kernel<D, kKind>, grid, PL::kThreads, PL::kSmem, st, a, list, units,
                      dense, map);
}

cudaError_t launch_chunk_tc(const ChunkArgs& a, const ChunkList& list, const ChunkUnits& units,
                            const DenseTiles& dense, const CUtensorMap& map, CacheKind kind,
                            bool fresh, cudaStream_t st) {
  if (a.g.D != 64 && a.g.D != 128) return cudaErrorInvalidValue;
  const bool wide = a.g.D == 128;
  switch (a.dense ? kUnfolded : kind) {
    case kCacheBf16:
      return wide ? run_tc<128, kCacheBf16>(a, list, units, dense, map, fresh, st)
                  : run_tc<64, kCacheBf16>(a, list, units, dense, map, fresh, st);
    case kCacheInt8:
      return wide ? run_tc<128, kCacheInt8>(a, list, units, dense, map, fresh, st)
                  : run_tc<64, kCacheInt8>(a, list, units, dense, map, fresh, st);
    case kCacheE4m3:
      return wide ? run_tc<128, kCacheE4m3>(a, list, units, dense, map, fresh, st)
                  : run_tc<64, kCacheE4m3>(a, list, units, dense, map, fresh, st);
    case kUnfolded:
      return wide ? run_tc<128, kUnfolded>(a, list, units, dense, map, fresh, st)
                  : run_tc<64, kUnfolded>(a, list, units, dense, map, fresh, st);
  }
  return cudaErrorInvalidValue;
}

}  // namespace td
