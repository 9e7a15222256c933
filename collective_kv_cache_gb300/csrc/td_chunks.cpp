// td_chunks.cpp - entry points over chunks of new tokens: 8-bit pages written and read back,
// attention of the chunks over bf16 or 8-bit pages. Validation and the launches' plans.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <new>
#include <vector>

#include "td_ctx.h"

using namespace td;

namespace {

constexpr int64_t kMaxPosition = INT32_MAX / 2;

bool cache_kind(int32_t format, CacheKind* kind) {
  if (format == TD_KV_INT8) *kind = kCacheInt8;
  else if (format == TD_KV_E4M3) *kind = kCacheE4m3;
  else return false;
  return true;
}

td_status pages_dev(const td_ctx* c, void* base, int64_t num_pages, const int32_t* table,
                    int32_t max_lp, PoolDev* out) {
  const int P = c->shape.page_size;
  // rows of a layer's K or V are numbered in 32 bits
  if (!base || !table || !aligned16(base) || num_pages < 1 || max_lp < 1 ||
      num_pages > INT32_MAX / P)
    return TD_ERR_INVALID_ARG;
  out->base = static_cast<uint16_t*>(base);
  out->num_pages = num_pages;
  out->bt = table;
  out->max_lp = max_lp;
  out->P = P;
  out->p_shift = is_pow2(P) ? log2i(P) : -1;
  return TD_OK;
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

bool layers_ok(const td_ctx* c, int32_t begin, int32_t end) {
  return begin >= 0 && end <= c->shape.n_layers && begin < end;
}

// The sequences [x0, x0 + list->n) of the call.
void fill_list(const td_chunks* ch, int x0, ChunkList* list) {
  list->n = std::min(ch->n - x0, kMaxChunkSeqs);
  list->row[0] = 0;
  for (int x = 0; x < list->n; ++x) {
    list->agent[x] = ch->agent[x0 + x];
    list->start[x] = ch->start[x0 + x];
    list->row[x + 1] = list->row[x] + ch->len[x0 + x];
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
  if (D > 256) return TD_ERR_INVALID_ARG;   // a warp holds a head row, 8 elements a lane
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
  a.lane_shift = log2i((D + 7) / 8);
  a.head_mul = ((1 << 20) + c->g.H - 1) / c->g.H;
  a.err = c->d_err;
  // tokens per CTA: 32, fewer where the grid would leave SMs without a CTA
  a.per_cta = kQuantTokens;
  while (a.per_cta > 4 &&
         (tokens + a.per_cta - 1) / a.per_cta * a.nl * 2 < 4 * static_cast<int64_t>(c->sm_count))
    a.per_cta >>= 1;
  int64_t tok0 = 0;
  for (int x0 = 0; x0 < ch->n; x0 += kMaxChunkSeqs) {
    ChunkList list;
    fill_list(ch, x0, &list);
    a.tok0 = tok0;
    const cudaError_t e = write ? launch_quantise(a, list, kind, st)
                                : launch_dequantise(a, list, kind, st);
    if (e != cudaSuccess) return TD_ERR_CUDA;
    tok0 += list.row[list.n];
  }
  return TD_OK;
}

// Scratch of at least `need` floats. An outgrown buffer stays until the context goes: a
// captured graph may hold its address. Inside a capture nothing can be allocated.
td_status chunk_scratch(td_ctx* c, size_t need, cudaStream_t st) {
  if (need <= c->chunk_cap) return TD_OK;
  if (capturing(st)) return TD_ERR_INVALID_ARG;
  const size_t cap = std::max(need, 2 * c->chunk_cap);
  float* p = nullptr;
  if (c->d_chunk) c->old_chunk.reserve(c->old_chunk.size() + 1);
  if (cudaMalloc(&p, cap * sizeof(float)) != cudaSuccess) {
    cudaGetLastError();
    return TD_ERR_CUDA;
  }
  if (c->d_chunk) c->old_chunk.push_back(c->d_chunk);
  c->d_chunk = p;
  c->chunk_cap = cap;
  return TD_OK;
}

td_status run_chunk_attention(td_ctx* c, const td_chunks* ch, const PoolDev& pool,
                              const float* scale8, CacheKind kind, int32_t layer_begin,
                              int32_t layer_end, const void* q, int32_t n_q_heads, float scale,
                              int32_t window, int32_t n_sink, void* out, float* lse,
                              cudaStream_t st) {
  const int H = c->g.H, D = c->g.D;
  if ((D != 64 && D != 128) || n_q_heads < H || n_q_heads % H != 0 || !std::isfinite(scale) ||
      window < 0 || n_sink < 0 || !layers_ok(c, layer_begin, layer_end))
    return TD_ERR_INVALID_ARG;
  int64_t tokens = 0;
  td_status s = check_chunks(c, ch, pool.max_lp, &tokens);
  if (s != TD_OK) return s;
  if (tokens == 0) return TD_OK;
  if (!q || !out || !aligned16(q) || !aligned16(out) ||
      (reinterpret_cast<uintptr_t>(lse) & 3u) != 0 || tokens > INT32_MAX / n_q_heads)
    return TD_ERR_INVALID_ARG;
  ChunkArgs a{};
  a.g = c->g;
  a.pool = pool;
  a.scale = scale8;
  a.q = static_cast<const uint16_t*>(q);
  a.out = static_cast<uint16_t*>(out);
  a.lse = lse;
  a.tokens = tokens;
  a.nq = n_q_heads;
  a.G = n_q_heads / H;
  a.nl = layer_end - layer_begin;
  a.layer_begin = layer_begin;
  a.window = window;
  a.n_sink = n_sink;
  a.scale_log2 = scale * 1.4426950408889634f;
  a.err = c->d_err;
  int64_t tok0 = 0;
  for (int x0 = 0; x0 < ch->n; x0 += kMaxChunkSeqs) {
    ChunkList list;
    fill_list(ch, x0, &list);
    a.tok0 = tok0;
    tok0 += list.row[list.n];
    if (list.row[list.n] == 0) continue;
    int most_rows = 0;
    for (int x = 0; x < list.n; ++x)
      most_rows = std::max(most_rows, (list.row[x + 1] - list.row[x]) * a.G);
    const int R = most_rows <= 8 ? 8 : 16;
    // visible positions of a tile of sequence x, at most
    auto seen = [&](int x) -> int64_t {
      const int64_t all = static_cast<int64_t>(list.start[x]) + list.row[x + 1] - list.row[x];
      return window == 0 ? all
                         : std::min<int64_t>(all, static_cast<int64_t>(window) + n_sink +
                                                      (R - 1) / a.G + 1);
    };
    auto tiles = [&](int x) -> int64_t {
      return (static_cast<int64_t>(list.row[x + 1] - list.row[x]) * a.G + R - 1) / R;
    };
    int64_t positions = 0, longest = 0;
    for (int x = 0; x < list.n; ++x) {
      if (tiles(x) == 0) continue;
      positions += tiles(x) * seen(x);
      longest = std::max(longest, seen(x));
    }
    const int64_t warps = static_cast<int64_t>(c->sm_count) * 12;
    int64_t span = positions * H * a.nl / warps;
    span = std::max<int64_t>((span + 15) / 16 * 16, 128);
    a.span = static_cast<int>(std::min<int64_t>(span, (longest + 15) / 16 * 16));
    ChunkUnits units;
    units.base[0] = 0;
    a.direct = 1;
    int64_t sum = 0;
    for (int x = 0; x < list.n; ++x) {
      const int64_t ns = std::max<int64_t>((seen(x) + a.span - 1) / a.span, 1);
      if (tiles(x) > 0 && ns > 1) a.direct = 0;
      sum += tiles(x) * ns;
      if (sum > INT32_MAX) return TD_ERR_INVALID_ARG;
      units.nsplit[x] = static_cast<int32_t>(ns);
      units.base[x + 1] = static_cast<int32_t>(sum);
    }
    const int64_t n = sum * H * a.nl;
    if (n > INT32_MAX) return TD_ERR_INVALID_ARG;
    if (!a.direct) {
      if ((s = chunk_scratch(c, static_cast<size_t>(n) * R * (D + 2), st)) != TD_OK) return s;
      a.part_o = c->d_chunk;
      a.part_ml = c->d_chunk + static_cast<size_t>(n) * R * D;
    }
    if (launch_chunk_rows(a, list, units, kind, R, st) != cudaSuccess ||
        (!a.direct && launch_chunk_join(a, list, units, R, st) != cudaSuccess))
      return TD_ERR_CUDA;
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
  return run_chunk_attention(c, ch, pd, nullptr, kCacheBf16, layer_begin, layer_end, q, n_q_heads,
                             scale, window, n_sink, out, lse, static_cast<cudaStream_t>(stream));
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
  return run_chunk_attention(c, ch, cd.pool, cd.scale, kind, layer_begin, layer_end, q, n_q_heads,
                             scale, window, n_sink, out, lse, static_cast<cudaStream_t>(stream));
} catch (const std::bad_alloc&) {
  return TD_ERR_CUDA;
}

}  // extern "C"
