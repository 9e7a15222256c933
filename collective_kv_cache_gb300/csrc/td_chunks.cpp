// td_chunks.cpp - entry points over chunks of new tokens: 8-bit pages written and read back,
// attention of the chunks over bf16, 8-bit or 4-bit pages. Validation and the launches' plans.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <memory>
#include <new>
#include <vector>

#include "td_ctx.h"

using namespace td;

namespace {

bool cache_kind(int32_t format, CacheKind* kind) {
  if (format == TD_KV_INT8) *kind = kCacheInt8;
  else if (format == TD_KV_E4M3) *kind = kCacheE4m3;
  else return false;
  return true;
}

td_status pages8_dev(const td_ctx* c, const td_paged8* p, Cache8Dev* out, CacheKind* kind) {
  if (!p || !p->scale || (reinterpret_cast<uintptr_t>(p->scale) & 3u) != 0 ||
      !cache_kind(p->format, kind))
    return TD_ERR_INVALID_ARG;
  out->scale = p->scale;
  return pages_dev(c, p->codes, p->num_pages, p->block_table, p->max_pages_per_agent, &out->pool);
}

// Checks the chunks against the context and the block table; *tokens = their sum.
td_status check_chunks(const td_ctx* c, const td_chunks* ch, int32_t max_lp, int64_t* tokens) {
  if (!ch || ch->n < 0 || (ch->n > 0 && (!ch->agent || !ch->start || !ch->len)))
    return TD_ERR_INVALID_ARG;
  const int64_t most = std::min<int64_t>(static_cast<int64_t>(max_lp) * c->shape.page_size,
                                         kMaxPosition);
  int64_t sum = 0;
  for (int x = 0; x < ch->n; ++x) {
    if (ch->agent[x] < 0 || ch->agent[x] >= c->max_agents || ch->start[x] < 0 || ch->len[x] < 0 ||
        static_cast<int64_t>(ch->start[x]) + ch->len[x] > most)
      return TD_ERR_INVALID_ARG;
    sum += ch->len[x];
  }
  *tokens = sum;
  return TD_OK;
}

// The list of the sequences order[*at], order[*at + 1], ... (at most kMaxChunkSeqs; *at moves
// past them). tok: the dense row of each sequence's first token.
void fill_list(const td_chunks* ch, const std::vector<int32_t>& order,
               const std::vector<int32_t>& tok, size_t* at, ChunkList* list) {
  list->n = 0;
  list->row[0] = 0;
  for (; *at < order.size() && list->n < kMaxChunkSeqs; ++*at) {
    const int x = order[*at], i = list->n++;
    list->tok[i] = tok[x];
    list->agent[i] = ch->agent[x];
    list->start[i] = ch->start[x];
    list->row[i + 1] = list->row[i] + ch->len[x];
  }
}

// The sequences that have tokens, in the batch's order, and every sequence's first dense row.
void sequences(const td_chunks* ch, std::vector<int32_t>* order, std::vector<int32_t>* tok) {
  order->reserve(ch->n);
  tok->reserve(ch->n);
  int32_t sum = 0;
  for (int x = 0; x < ch->n; ++x) {
    tok->push_back(sum);
    sum += ch->len[x];
    if (ch->len[x] > 0) order->push_back(x);
  }
}

// No position of an agent may be written by two of the chunks.
bool chunks_disjoint(const td_chunks* ch) {
  std::vector<int32_t> order(ch->n);
  int m = 0;
  for (int x = 0; x < ch->n; ++x)
    if (ch->len[x] > 0) order[m++] = x;
  std::sort(order.begin(), order.begin() + m, [&](int32_t a, int32_t b) {
    return ch->agent[a] != ch->agent[b] ? ch->agent[a] < ch->agent[b] : ch->start[a] < ch->start[b];
  });
  for (int i = 1; i < m; ++i) {
    const int a = order[i - 1], b = order[i];
    if (ch->agent[a] == ch->agent[b] && ch->start[a] + ch->len[a] > ch->start[b]) return false;
  }
  return true;
}

td_status run_quant(td_ctx* c, const td_chunks* ch, const td_paged8* cache, const void* k,
                    const void* v, int32_t layer_begin, int32_t layer_end, bool write,
                    cudaStream_t st) {
  if (!c || !same_device(c) || !cache || !layers_ok(c, layer_begin, layer_end))
    return TD_ERR_INVALID_ARG;
  const int D = c->g.D;
  if (D > 256) return TD_ERR_INVALID_ARG;   // (a warp would hold a head row of 512)
  QuantArgs a{};
  CacheKind kind;
  td_status s = pages8_dev(c, cache, &a.cache, &kind);
  if (s != TD_OK) return s;
  int64_t tokens = 0;
  if ((s = check_chunks(c, ch, cache->max_pages_per_agent, &tokens)) != TD_OK) return s;
  if (tokens > INT32_MAX / 2) return TD_ERR_INVALID_ARG;
  if (tokens == 0) return TD_OK;
  if (!k || !v || !aligned16(k) || !aligned16(v)) return TD_ERR_INVALID_ARG;
  if (write && !chunks_disjoint(ch)) return TD_ERR_INVALID_ARG;
  a.g = c->g;
  a.k = static_cast<uint16_t*>(const_cast<void*>(k));
  a.v = static_cast<uint16_t*>(const_cast<void*>(v));
  a.tokens = tokens;
  a.nl = layer_end - layer_begin;
  a.layer_begin = layer_begin;
  a.lane_shift = log2i(write ? D / 16 : D / 8);
  a.head_mul = ((1 << 20) + c->g.H - 1) / c->g.H;
  a.err = c->d_err;
  // tokens per CTA: 32, fewer where the grid would leave SMs without a CTA
  a.per_cta = kQuantTokens;
  while (a.per_cta > 4 &&
         (tokens + a.per_cta - 1) / a.per_cta * a.nl * 2 < 4 * static_cast<int64_t>(c->sm_count))
    a.per_cta >>= 1;
  std::vector<int32_t> order, tok;
  sequences(ch, &order, &tok);
  for (size_t at = 0; at < order.size();) {
    ChunkList list;
    a.tok0 = tok[order[at]];
    fill_list(ch, order, tok, &at, &list);
    const cudaError_t e = write ? launch_quantise(a, list, kind, st)
                                : launch_dequantise(a, list, kind, st);
    if (e != cudaSuccess) return TD_ERR_CUDA;
  }
  return TD_OK;
}

// Query rows of a sequence (per kv head) up to which the streaming kernel takes it. One more and
// it would read the pages twice over: 28 rows on 4000 to 6000 positions of 32 agents take 66 us
// on the tensor-core kernel and 143 on the streaming one (D = 128; 44 and 87 at D = 64), 56 rows 67
// and 271, 30 rows on 1000 positions 17 and 32. Over 8-bit pages two passes come out even: 28 rows
// 117 and 119 us over int8, 118 and 114 over e4m3 (D = 64: 90 and 78, 78 and 72; 30 rows on 1000
// positions 26 and 28, 24 and 27), 56 rows 117 and 218. Up to 16 rows the tensor-core kernel's
// tile of 128 is mostly empty. Over 4-bit pages the streaming kernel is bound by its instructions
// and the other by converting the codes, which more rows share: 28 rows on 5000 positions of 32
// agents take 56 us streamed and 91 on the tensor-core kernel (int4, 4 kv heads, D = 128; e2m1 61 and
// 96), 48 rows 77 and 91 (84 and 96), 56 rows 98 and 91 (107 and 96); at D = 64 38 and 70 (41 and 69), 52
// and 70 (56 and 71), 67 and 70 (72 and 71). On 1000 positions of 8 agents 48 rows 13.1 and 16.3 (13.3 and
// 15.3; 10.0 and 13.9, 10.2 and 12.9), 56 rows 13.9 and 16.8 (14.4 and 15.8; 10.9 and 14.4, 11.3 and 13.3).
constexpr int kFewRows = 16;
constexpr int kFewRows4 = 48;

// Over 8-bit pages the tensor-core kernel converts the codes itself for up to two tiles of query
// rows (of 256); from three on they are unfolded once, before it. Two tiles of 480 rows on 12000
// positions of 16 agents take 259 us converted in the kernel and 269 unfolded (int8, 4 kv heads,
// D = 128; 2000 positions of 8: 42.5 and 43.4; e4m3 242 and 260), 960 rows 564 and 420 (53 and 46;
// 529 and 403), 2560 rows 1093 and 795 (129 and 104; 1021 and 735). At D = 64 the crossing is the
// same. Over 4-bit pages it is too where all sequences are of two tiles at most (480 rows on 12000
// positions of 16 agents 237 us converted in the kernel and 263 unfolded, e2m1 225 and 242; one tile
// of 112 rows 92 and 152 to 162). Where longer ones are unfolded all the same, those of two tiles go
// with them, which spares a launch its long last units: 32 spans of 5 to 1505 rows 950 us, and
// 970 with two tiles converted (int4 1028 and 1037).
constexpr int kOwnRows = 512;
// The unfolded copy of one launch, at most: sequences that would pass it go to the next one, a
// sequence that is longer by itself is converted in the kernel.
constexpr int64_t kDenseBytes = int64_t{1} << 30;
// The copy of sequences that are unfolded beside longer ones instead of streamed, or of being converted
// in the kernel, at most: written in 6 us, some launch's time, and 25, as long as their conversion.
constexpr int64_t kJoinBytes[2] = {int64_t{1} << 25, int64_t{1} << 27};

// KV tiles of sequence x's unfolded copy, and a tile's bytes over the call's layers.
int64_t dense_tiles(const td_chunks* ch, int x, const ChunkArgs& a) {
  return dense_span(ch->start[x], ch->len[x], a.window, a.n_sink).n;
}
int64_t dense_tile_bytes(const ChunkArgs& a) {
  return static_cast<int64_t>(a.nl) * 2 * 128 * (a.g.E * 2 + a.g.H * 4);
}

// The first tiles of the list's sequences; those that do not fit go back to the order.
void fill_dense(const td_chunks* ch, const std::vector<int32_t>& order, const ChunkArgs& a,
                size_t* at, ChunkList* list, DenseTiles* dense) {
  const int64_t most = kDenseBytes / dense_tile_bytes(a);
  const size_t first = *at - list->n;
  int64_t sum = 0;
  int n = 0;
  dense->base[0] = 0;
  for (; n < list->n; ++n) {
    sum += dense_tiles(ch, order[first + n], a);
    if (sum > most) break;
    dense->base[n + 1] = static_cast<int32_t>(sum);
  }
  *at -= list->n - n;
  list->n = n;
}

// The bf16 pages of the call's layers as a tensor map of boxes that lie inside a page; false
// where the tensor-core kernel cannot read them: pages that are no multiple of 8 tokens (a
// box is at least 8 rows, the period of the swizzle), or more rows than a coordinate counts.
bool row_map(int E, uint16_t* base, int64_t rows, int b, CUtensorMap* m);
bool bf16_map(const td_ctx* c, const ChunkArgs& a, const PoolDev& pool, int* box, CUtensorMap* m) {
  if (pool.P % 8 != 0) return false;
  const int64_t plane = pool.num_pages * pool.P;
  const int64_t rows = 2 * plane * a.nl;
  if (rows > INT32_MAX) return false;
  int b = 8;
  while (b < 128 && pool.P % (2 * b) == 0) b *= 2;
  *box = b;
  const int E = c->g.E;
  return row_map(E, pool.base + static_cast<int64_t>(a.layer_begin) * 2 * plane * E, rows, b, m);
}

// Rows of E bf16 as a tensor map of boxes of b rows x 64.
bool row_map(int E, uint16_t* base, int64_t rows, int b, CUtensorMap* m) {
  EncodeTiledFn fn = encode_tiled();
  if (!fn) return false;
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(E), static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(E) * 2};
  const cuuint32_t bx[2] = {64, static_cast<cuuint32_t>(b)};
  const cuuint32_t elem[2] = {1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT16, 2, base, dims, strides, bx, elem,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) ==
         CUDA_SUCCESS;
}

// Sequences' tiles of query rows, and the steps of positions that one of them sees at most.
struct Loads {
  uint32_t tiles[kMaxChunkSeqs], seen[kMaxChunkSeqs];
};

// Cuts every tile's visible positions (in steps of `step` positions) into parts of one length
// and fills base, nsplit, span and direct; the number of units, or -1. The length is the one
// with the least estimated time among the divisions of the longest tile.
struct Cost {
  int64_t slots;      // units that run at once
  int64_t heads;      // kv heads x layers
  double step_us;     // a step of a unit, with the others beside it
  double fixed_us;    // what a unit costs besides its steps
  double step_bytes;  // that a step reads, at 6.5 TB/s for all units together
  int least;          // steps per unit, at least
  double row_bytes;   // of partial results per part, over all rows of the launch
};

int64_t cut(const ChunkList& list, const Cost& cost, const Loads& loads, int step, ChunkArgs* a,
            ChunkUnits* units) {
  const uint32_t* const seen = loads.seen;
  int64_t longest = 1, total = 0;
  for (int x = 0; x < list.n; ++x) {
    longest = std::max<int64_t>(longest, seen[x]);
    total += static_cast<int64_t>(loads.tiles[x]) * seen[x];
  }
  int64_t best = longest, last = 0;
  double best_us = 0.0;
  for (int64_t k = 1; k <= 256; k = k < 16 ? k + 1 : k + k / 8) {
    const int64_t span = std::max<int64_t>((longest + k - 1) / k,
                                           std::min<int64_t>(cost.least, longest));
    if (span == last) continue;
    last = span;
    int64_t n = 0;
    const uint32_t s32 = static_cast<uint32_t>(span);
    for (int x = 0; x < list.n; ++x)
      n += static_cast<int64_t>(loads.tiles[x]) * ((seen[x] + s32 - 1) / s32);
    const int64_t most = (longest + span - 1) / span;
    n *= cost.heads;
    // one wave: its longest unit; more: the slots' share of the work and half a unit of tail;
    // or the bytes
    const double unit = span * cost.step_us + cost.fixed_us;
    const double work = static_cast<double>(total) * cost.heads;
    double us = n <= cost.slots
                    ? unit
                    : std::max(unit, (work * cost.step_us + n * cost.fixed_us) / cost.slots + unit / 2);
    us = std::max(us, work * cost.step_bytes / 6.5e6);
    // joining: a launch, and the parts written and read once
    if (most > 1) us += 4.0 + 2.0 * cost.row_bytes * most / 5e6;
    if (k == 1 || us < best_us) {
      best_us = us;
      best = span;
    }
    if (span <= cost.least) break;
  }
  a->span = static_cast<int>(best * step);
  a->direct = 1;
  a->whole_units = a->join_from = 0;
  units->base[0] = 0;
  int64_t sum = 0;
  for (int x = 0; x < list.n; ++x) {
    const int64_t ns = (seen[x] + best - 1) / best;
    if (ns > 1) a->direct = 0;
    sum += loads.tiles[x] * ns;
    if (sum > INT32_MAX) return -1;
    units->nsplit[x] = static_cast<int32_t>(ns);
    units->whole[x] = 0;
    units->base[x + 1] = static_cast<int32_t>(sum);
  }
  return sum * cost.heads > INT32_MAX ? -1 : sum * cost.heads;
}

// Where every tile is one unit and they are one to six waves of the machine: the tiles of the
// last, partly filled wave are cut into parts that fill it, where that is estimated to gain
// more than their join costs. The order is the launch's: sequences from first to last. 156
// units of one sequence: 142 us whole, 103 with the last 4 in eight parts; 376 (chunks of 500 to
// 700 tokens over e4m3 pages, the last 72 in halves) 276 and 261, but 278 in thirds, which are
// more than one wave again. 984 units of unequal length (6.5 waves) fill the machine by
// themselves: 724 us whole, 733 cut.
int64_t cut_tail(const ChunkList& list, const Cost& cost, const Loads& loads, int64_t n,
                 double unit_bytes, ChunkArgs* a, ChunkUnits* units) {
  const int64_t r = n % cost.slots;
  if (!a->direct || n <= cost.slots || n > 6 * cost.slots || r == 0) return n;
  const int64_t m = (r + cost.heads - 1) / cost.heads;      // the tail's tiles
  double total = 0.0, tail = 0.0;
  int64_t left = m, longest = 0;                            // steps of the tail's first unit
  for (int x = list.n - 1; x >= 0; --x) {
    const double us = (loads.seen[x] * cost.step_us + cost.fixed_us) * cost.heads;
    total += loads.tiles[x] * us;
    const int64_t take = std::min<int64_t>(left, loads.tiles[x]);
    if (take > 0) longest = loads.seen[x];
    tail += take * us;
    left -= take;
  }
  const double full = (total - tail) / cost.slots;
  double best_us = 0.97 * (full + longest * cost.step_us + cost.fixed_us);
  int64_t best = 0;
  for (int64_t k = 2; k <= 8 && longest / k >= cost.least; ++k) {
    const double part = (longest + k - 1) / k * cost.step_us + cost.fixed_us;
    const int64_t waves = (m * cost.heads * k + cost.slots - 1) / cost.slots;
    const double us =
        full + waves * part + 4.0 + 2.0 * m * cost.heads * k * unit_bytes / 10e6;
    if (us < best_us) {
      best_us = us;
      best = k;
    }
  }
  if (best == 0) return n;
  const int64_t span = (longest + best - 1) / best;
  a->span = static_cast<int>(span);
  a->direct = 0;
  left = m;
  for (int x = list.n - 1; x >= 0; --x) {
    const int64_t take = std::min<int64_t>(left, loads.tiles[x]);
    left -= take;
    units->whole[x] = static_cast<int32_t>(loads.tiles[x] - take);
    units->nsplit[x] = take ? static_cast<int32_t>((loads.seen[x] + span - 1) / span) : 1;
    if (take) a->join_from = list.row[x];
  }
  int64_t sum = 0;
  bool whole = true;
  for (int x = 0; x < list.n; ++x) {
    units->base[x] = static_cast<int32_t>(sum);
    if (whole) a->whole_units = static_cast<int>(sum + units->whole[x]);
    const int64_t cut = static_cast<int64_t>(loads.tiles[x]) - units->whole[x];
    whole = whole && cut == 0;
    sum += units->whole[x] + cut * units->nsplit[x];
  }
  units->base[list.n] = static_cast<int32_t>(sum);
  return sum * cost.heads;
}

// Positions that a tile of `rows` query rows of sequence x sees, at most.
int64_t seen_positions(const ChunkList& list, const ChunkArgs& a, int x, int rows) {
  const int64_t all = static_cast<int64_t>(list.start[x]) + list.row[x + 1] - list.row[x];
  if (a.window == 0) return all;
  return std::min<int64_t>(all, static_cast<int64_t>(a.window) + a.n_sink + (rows - 1) / a.G + 1);
}

uint32_t tiles_of(const ChunkList& list, const ChunkArgs& a, int x, int rows) {
  const int64_t all = static_cast<int64_t>(list.row[x + 1] - list.row[x]) * a.G;
  return static_cast<uint32_t>((all + rows - 1) / rows);
}

// Bytes of one part of every query row's partial result.
double partial_bytes(const ChunkList& list, const ChunkArgs& a) {
  return 4.0 * (a.g.D + 2) * a.nl * a.nq * list.row[list.n];
}

int64_t plan_rows(const td_ctx* c, const ChunkList& list, ChunkArgs* a, ChunkUnits* units,
                  int* rows) {
  int64_t most = 0;
  for (int x = 0; x < list.n; ++x)
    most = std::max<int64_t>(most, static_cast<int64_t>(list.row[x + 1] - list.row[x]) * a->G);
  const int R = *rows = most <= 8 ? 8 : 16;
  // three blocks an SM (two with 16 rows a tile); a step of 128 positions of the block's four
  // warps took 3.1 us in bf16 at D = 128, 2 us otherwise, with all blocks in place
  const int64_t slots = static_cast<int64_t>(c->sm_count) * (R == 8 ? 3 : 2);
  const double bytes = 2.0 * 128 * a->g.D * (a->scale ? 1 : 2);
  const Cost cost{slots, static_cast<int64_t>(a->g.H) * a->nl,
                  !a->scale && a->g.D == 128 ? 3.1 : 2.0, 4.0, bytes, 2, partial_bytes(list, *a)};
  Loads loads;
  for (int x = 0; x < list.n; ++x) {
    loads.tiles[x] = tiles_of(list, *a, x, R);
    loads.seen[x] = static_cast<uint32_t>((seen_positions(list, *a, x, R) + 127) / 128);
  }
  return cut(list, cost, loads, 128, a, units);
}

// The same over 4-bit pages, whose blocks share the steps evenly.
int64_t plan_rows4(const td_ctx* c, const ChunkList& list, ChunkArgs* a, ChunkUnits* units,
                   int* rows) {
  int64_t most = 0;
  for (int x = 0; x < list.n; ++x)
    most = std::max<int64_t>(most, static_cast<int64_t>(list.row[x + 1] - list.row[x]) * a->G);
  const int R = *rows = most <= 8 ? 8 : 16;
  const int64_t heads = static_cast<int64_t>(a->g.H) * a->nl;
  const int target = cut_target(static_cast<int64_t>(c->sm_count) * token4_blocks(R, c->g.D), heads);
  int64_t total = 0, tiles = 0;
  for (int x = 0; x < list.n; ++x) {
    units->whole[x] = static_cast<int32_t>(tiles);
    units->nsplit[x] = static_cast<int32_t>((seen_positions(list, *a, x, R) + 127) / 128);
    tiles += tiles_of(list, *a, x, R);
    total += static_cast<int64_t>(units->nsplit[x]) * tiles_of(list, *a, x, R);
    if (total > INT32_MAX || tiles > INT32_MAX) return -1;
  }
  if ((target + tiles) * heads > INT32_MAX) return -1;
  a->cut = cut_steps(total, tiles, target, static_cast<int>(target + tiles));
  const int64_t share = a->cut.share;
  int64_t begin = 0;
  a->direct = 1;
  units->base[0] = 0;
  for (int x = 0; x < list.n; ++x) {
    const int64_t places = tile_places(a->cut.crossing, share, units->nsplit[x]);
    if (places > 1) a->direct = 0;
    begin += tiles_of(list, *a, x, R) * places;
    if (begin > INT32_MAX / 2) return -1;
    units->base[x + 1] = static_cast<int32_t>(begin);
  }
  a->cut.blocks = static_cast<int>(a->cut.crossing ? (begin + share - 1) / share : begin);
  return a->cut.units * heads;
}

int64_t plan_tc(const td_ctx* c, const ChunkList& list, ChunkArgs* a, ChunkUnits* units,
                int* rows) {
  int64_t most = 0;
  for (int x = 0; x < list.n; ++x)
    most = std::max<int64_t>(most, static_cast<int64_t>(list.row[x + 1] - list.row[x]) * a->G);
  // 4-bit pages: where few units see little, tiles of 128 rows too, twice the units. On long contexts
  // the conversion is the bound, and is made twice: 8 sequences of 252 rows (int4, D = 128, in graphs) on
  // 500 positions 18.5 us in tiles of 256 and 16.0 in tiles of 128, on 1000 27.6 and 23.8, on 2000 35.7 and
  // 39.3, on 2400, past the limit, 37.3 and 42.6, on 6000 55 and 70; e2m1 and D = 64 cross at the same
  // place. Unfolded, 2 of 1050 rows: on 1000 23.5 and 18.0, on 5000 44 and 37, past the limit on 5800 48
  // and 40, on 9000 63 and 53.
  bool small = most <= 128;
  if (a->word && !small) {
    int64_t n = 0, steps = 0;
    for (int x = 0; x < list.n; ++x) {
      const int64_t here = tiles_of(list, *a, x, 256) * static_cast<int64_t>(a->g.H) * a->nl;
      n += here;
      steps += here * ((seen_positions(list, *a, x, 256) + 127) / 128);
    }
    small = 2 * n <= c->sm_count && steps <= (a->dense_rows ? 12 : 4) * c->sm_count;
  }
  const int R = *rows = a->rows_cta = small ? 128 : 256;
  // one CTA an SM; a KV tile's products and softmax
  const bool codes = a->scale && !a->dense_rows;
  // (unfolded 4-bit pages in tiles of 128 rows: two KV tiles at a time. Taken for as long as the others,
  // 8 chunks of 7 to 840 rows on 500 to 1500 positions were cut, and took 24.9 us instead of 19.4)
  const bool turns = a->word && a->dense_rows && R == 128;
  const double step = codes ? 2.4 : (a->g.D == 128 ? 1.4 : 0.8) * (turns ? 0.6 : 1.0);
  const Cost cost{c->sm_count, static_cast<int64_t>(a->g.H) * a->nl, step, 4.0,
                  2.0 * 128 * a->g.D * (codes ? 1 : 2) / 8, 2, partial_bytes(list, *a)};
  Loads loads;
  for (int x = 0; x < list.n; ++x) {
    loads.tiles[x] = tiles_of(list, *a, x, R);
    int64_t all =
        (static_cast<int64_t>(list.start[x]) + list.row[x + 1] - list.row[x] + 127) / 128;
    // a window's positions may straddle one tile more, the first ones' another
    if (a->window) all = std::min(all, (seen_positions(list, *a, x, R) + 127) / 128 + 2);
    loads.seen[x] = static_cast<uint32_t>(all);
  }
  const int64_t n = cut(list, cost, loads, 1, a, units);
  return n < 0 ? n : cut_tail(list, cost, loads, n, 4.0 * R * (a->g.D + 2), a, units);
}

// 4-bit pages: a kind of few sequences joins the next one's launch, where that costs less than a
// launch of its own. Unfolded (order[2]) are also the others whose copies are small; the tensor-core
// kernel (order[1]) also takes streamed ones (order[0]) of few KV tiles, where all units run at once.
// 24 chunks of 7 to 700 rows on 2000 to 2500 positions 102 us in three kinds, 76 joined; 8 of 7 to
// 840 on 500 to 1500 41 and 28; 46 of 42 and 49 on 20 to 110 14.3 and 7.4. The streamed ones' limit: 16 of 7
// to 140 rows (int4, D = 128, in graphs) on 500 positions take 17 us joined and 33 apart, on 1000 23 and
// 35, on 2000, past it, 39 and 44, on 3000 53 and 50, on 4000 65 and 60 (e2m1 36 and 42, 50 and 48, 64 and
// 58; D = 64 31 and 37, 44 and 42, 55 and 48).
void join_orders(const td_ctx* c, const td_chunks* ch, const ChunkArgs& a, int64_t longest,
                 int64_t most_tiles, std::vector<int32_t>* order) {
  auto move = [&](int from, int to) {
    order[to].insert(order[to].end(), order[from].begin(), order[from].end());
    order[from].clear();
  };
  if (!order[2].empty()) {
    for (int from = 1; from >= 0; --from) {
      int64_t tiles = 0;
      for (const int32_t x : order[from]) tiles += dense_tiles(ch, x, a);
      if (tiles <= most_tiles && tiles * dense_tile_bytes(a) <= kJoinBytes[from]) move(from, 2);
    }
  }
  if (order[0].empty() || order[1].empty()) return;
  const int64_t R = longest <= 128 ? 128 : 256, heads = static_cast<int64_t>(a.g.H) * a.nl;
  int64_t units = 0, steps = 0;               // steps: of the streamed ones
  for (int i = 0; i < 2; ++i)
    for (const int32_t x : order[i]) {
      const int64_t n = (static_cast<int64_t>(ch->len[x]) * a.G + R - 1) / R * heads;
      units += n;
      if (i == 0) steps += n * dense_tiles(ch, x, a);
    }
  if (units <= c->sm_count && steps <= 2 * c->sm_count) move(0, 1);
}

td_status run_chunk_attention(td_ctx* c, const td_chunks* ch, const PoolDev& pool,
                              const float* scale8, const uint32_t* word4, CacheKind kind,
                              int32_t layer_begin,
                              int32_t layer_end, const void* q, int32_t n_q_heads, float scale,
                              int32_t window, int32_t n_sink, void* out, float* lse,
                              cudaStream_t st) {
  const int H = c->g.H, D = c->g.D;
  const float scale_log2 = scale * 1.4426950408889634f;
  if ((D != 64 && D != 128) || n_q_heads < H || n_q_heads % H != 0 || !std::isfinite(scale_log2) ||
      window < 0 || n_sink < 0 || !layers_ok(c, layer_begin, layer_end))
    return TD_ERR_INVALID_ARG;
  int64_t tokens = 0;
  td_status s = check_chunks(c, ch, pool.max_lp, &tokens);
  if (s != TD_OK) return s;
  if (tokens == 0) return TD_OK;
  if (!q || !out || !aligned16(q) || !aligned16(out) ||
      (reinterpret_cast<uintptr_t>(lse) & 3u) != 0 ||
      tokens > INT32_MAX / n_q_heads / (layer_end - layer_begin))
    return TD_ERR_INVALID_ARG;
  ChunkArgs a{};
  CUtensorMap map{};
  a.g = c->g;
  a.pool = pool;
  a.scale = scale8;
  a.word = word4;
  a.q = static_cast<const uint16_t*>(q);
  a.out = static_cast<uint16_t*>(out);
  a.lse = lse;
  a.tokens = tokens;
  a.nq = n_q_heads;
  a.G = n_q_heads / H;
  a.nl = layer_end - layer_begin;
  a.layer_begin = layer_begin;
  // (a window past every position is none; the kernels subtract it from positions)
  a.window = window > kMaxPosition ? 0 : window;
  a.n_sink = static_cast<int>(std::min<int64_t>(n_sink, kMaxPosition));
  a.scale_log2 = scale_log2;
  a.err = c->d_err;
  // Sequences of at most kFewRows query rows per kv head go to the streaming kernel, the
  // others to the tensor-core kernel, those of many rows over pages of codes by way of the
  // unfolded copy; each in lists of kMaxChunkSeqs. Plans first, so that the scratch is there
  // (or the call refused) before anything is launched.
  std::vector<int32_t> all, tok, order[3];
  sequences(ch, &all, &tok);
  const int few = four_bits(kind) ? kFewRows4 : kFewRows;
  int64_t longest = 0;
  for (const int32_t x : all) longest = std::max(longest, static_cast<int64_t>(ch->len[x]) * a.G);
  const int own = four_bits(kind) && longest > kOwnRows ? kOwnRows / 2 : kOwnRows;
  bool many = longest > few;
  if (many && kind == kCacheBf16) many = bf16_map(c, a, pool, &a.box_rows, &map);
  const int64_t most_tiles =
      kind != kCacheBf16 && encode_tiled() ? kDenseBytes / dense_tile_bytes(a) : 0;
  for (const int32_t x : all) {
    const int64_t rows = static_cast<int64_t>(ch->len[x]) * a.G;
    order[!many || rows <= few                                ? 0
          : rows <= own || dense_tiles(ch, x, a) > most_tiles ? 1
                                                              : 2].push_back(x);
  }
  if (four_bits(kind)) join_orders(c, ch, a, longest, most_tiles, order);
  // the longest contexts first: a unit of the tensor-core kernel takes an SM for as long as its
  // context is long, and the last ones to start should be short
  for (int i = 1; i < 3; ++i)
    std::stable_sort(order[i].begin(), order[i].end(), [&](int32_t x, int32_t y) {
      return ch->start[x] + ch->len[x] > ch->start[y] + ch->len[y];
    });
  a.tx_pad = c->attn_tx_pad;
  struct Launch {
    ChunkList list;
    ChunkUnits units;
    DenseTiles dense;
    ChunkArgs a;
    int group, rows;
    size_t planes, scales, parts, part_rows;
  };
  std::vector<std::unique_ptr<Launch>> launches;
  size_t need = 0;
  for (int group = 0; group < 3; ++group) {
    for (size_t at = 0; at < order[group].size();) {
      launches.emplace_back(new Launch);
      Launch& l = *launches.back();
      l.a = a;
      l.group = group;
      fill_list(ch, order[group], tok, &at, &l.list);
      if (group == 2) {
        fill_dense(ch, order[group], a, &at, &l.list, &l.dense);
        l.a.dense_rows = l.dense.base[l.list.n] * 128;
      }
      const int64_t n = group ? plan_tc(c, l.list, &l.a, &l.units, &l.rows)
                      : four_bits(kind) ? plan_rows4(c, l.list, &l.a, &l.units, &l.rows)
                                        : plan_rows(c, l.list, &l.a, &l.units, &l.rows);
      if (n < 0) return TD_ERR_INVALID_ARG;
      // the unfolded rows, their scales, then the partial results
      l.planes = static_cast<size_t>(a.nl) * 2 * l.a.dense_rows;
      l.scales = l.planes * a.g.E / 2;
      l.parts = l.scales + l.planes * H;
      l.part_rows =
          static_cast<size_t>(n - static_cast<int64_t>(l.a.whole_units) * H * a.nl) * l.rows;
      need = std::max(need, l.parts + (l.a.direct ? 0 : l.part_rows * (D + 2)));
    }
  }
  const size_t more = std::min(2 * c->chunk.cap, need + kScratchSpare);
  if ((s = grow(c, &c->chunk, need, more, st)) != TD_OK) return s;
  for (const auto& next : launches) {
    Launch& l = *next;
    l.a.part_o = c->chunk.p + l.parts;
    l.a.part_ml = l.a.direct ? nullptr : l.a.part_o + l.part_rows * D;
    if (l.group == 2) {
      l.a.dense = reinterpret_cast<uint16_t*>(c->chunk.p);
      l.a.dense_scale = c->chunk.p + l.scales;
      if (!row_map(a.g.E, l.a.dense, static_cast<int64_t>(l.planes), 128, &map) ||
          launch_expand(l.a, l.list, l.dense, kind, st) != cudaSuccess)
        return TD_ERR_CUDA;
    }
    const int first_bit = four_bits(kind) ? 10 + (kind - kCacheInt4) * 3 : kind * 3;
    const uint32_t bit = 1u << (l.group == 2 ? (four_bits(kind) && l.rows == 128 ? 20 : 9)
                                             : first_bit + (l.group ? 2 : l.rows == 8));
    const bool fresh = !(c->chunk_launched & bit);
    if ((l.group ? launch_chunk_tc(l.a, l.list, l.units, l.dense, map, kind, fresh, st)
                 : launch_chunk_rows(l.a, l.list, l.units, kind, l.rows, fresh, st)) !=
            cudaSuccess ||
        (!l.a.direct && launch_chunk_join(l.a, l.list, l.units, l.rows, st) != cudaSuccess))
      return TD_ERR_CUDA;
    c->chunk_launched |= bit;
  }
  return TD_OK;
}

}  // namespace

extern "C" {

td_status td_quantise_append(td_ctx* c, const td_chunks* ch, const td_paged8* cache,
                             const void* k_new, const void* v_new, int32_t layer_begin,
                             int32_t layer_end, void* stream) try {
  return run_quant(c, ch, cache, k_new, v_new, layer_begin, layer_end, true,
                   static_cast<cudaStream_t>(stream));
} catch (const std::bad_alloc&) {
  return TD_ERR_CUDA;
}

td_status td_dequantise_read(td_ctx* c, const td_chunks* ch, const td_paged8* cache,
                             int32_t layer_begin, int32_t layer_end, void* k_out, void* v_out,
                             void* stream) try {
  return run_quant(c, ch, cache, k_out, v_out, layer_begin, layer_end, false,
                   static_cast<cudaStream_t>(stream));
} catch (const std::bad_alloc&) {
  return TD_ERR_CUDA;
}

td_status td_chunk_attention(td_ctx* c, const td_chunks* ch, const td_paged* pool,
                             int32_t layer_begin, int32_t layer_end, const void* q,
                             int32_t n_q_heads, float scale, int32_t window, int32_t n_sink,
                             void* out, float* lse, void* stream) try {
  if (!c || !same_device(c) || !pool) return TD_ERR_INVALID_ARG;
  PoolDev pd;
  const td_status s = pages_dev(c, pool->base, pool->num_pages, pool->block_table,
                                pool->max_pages_per_agent, &pd);
  if (s != TD_OK) return s;
  return run_chunk_attention(c, ch, pd, nullptr, nullptr, kCacheBf16, layer_begin, layer_end, q,
                             n_q_heads, scale, window, n_sink, out, lse,
                             static_cast<cudaStream_t>(stream));
} catch (const std::bad_alloc&) {
  return TD_ERR_CUDA;
}

td_status td_chunk_attention_q8(td_ctx* c, const td_chunks* ch, const td_paged8* cache,
                                int32_t layer_begin, int32_t layer_end, const void* q,
                                int32_t n_q_heads, float scale, int32_t window, int32_t n_sink,
                                void* out, float* lse, void* stream) try {
  if (!c || !same_device(c) || !cache) return TD_ERR_INVALID_ARG;
  Cache8Dev cd;
  CacheKind kind;
  const td_status s = pages8_dev(c, cache, &cd, &kind);
  if (s != TD_OK) return s;
  return run_chunk_attention(c, ch, cd.pool, cd.scale, nullptr, kind, layer_begin, layer_end, q,
                             n_q_heads, scale, window, n_sink, out, lse,
                             static_cast<cudaStream_t>(stream));
} catch (const std::bad_alloc&) {
  return TD_ERR_CUDA;
}

td_status td_chunk_attention_q4(td_ctx* c, const td_chunks* ch, const td_paged4* cache,
                                int32_t layer_begin, int32_t layer_end, const void* q,
                                int32_t n_q_heads, float scale, int32_t window, int32_t n_sink,
                                void* out, float* lse, void* stream) try {
  if (!c || !same_device(c) || !cache) return TD_ERR_INVALID_ARG;
  Cache4Dev cd;
  CacheKind kind;
  const td_status s = pages4_dev(c, cache, &cd, &kind);
  if (s != TD_OK) return s;
  return run_chunk_attention(c, ch, cd.pool, nullptr, cd.word, kind, layer_begin, layer_end, q,
                             n_q_heads, scale, window, n_sink, out, lse,
                             static_cast<cudaStream_t>(stream));
} catch (const std::bad_alloc&) {
  return TD_ERR_CUDA;
}

}  // extern "C"
