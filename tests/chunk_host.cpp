// chunk_host.cpp - the chunk entry points (td_chunks.cpp) on a host without a GPU: the CUDA
// runtime calls and the kernel launches are stand-ins that record what they were given, so
// that refusals and launch plans can be tested by tests/test_chunks_host.py.
#include <cstdlib>
#include <map>
#include <vector>

#include "td_ctx.h"

using namespace td;

namespace {
struct Launch {
  int what;           // 0 quantise, 1 dequantise, 2 streaming attention, 3 join, 4 tensor cores
  int kind, rows;
  ChunkArgs a;
  QuantArgs qa;
  ChunkList list;
  ChunkUnits units;
  DenseTiles dense;
};
std::vector<Launch> g_launches;
struct Unfold {
  int before;         // the launch that follows
  int n;
  const uint16_t* to;
  int rows;
  DenseTiles dense;
};
std::vector<Unfold> g_unfolds;
int g_device = 0, g_capturing = 0, g_fail_malloc = 0;
size_t g_floats = 0, g_room = SIZE_MAX;
std::map<void*, size_t> g_held;      // what cudaMalloc gave and cudaFree has not had
bool g_synchronised = false, g_fail_wait = false;

Launch& push(int what, const ChunkList& list) {
  g_launches.emplace_back();
  Launch& l = g_launches.back();
  l.what = what;
  l.list = list;
  return l;
}
}  // namespace

namespace td {
cudaError_t launch_quantise(const QuantArgs& a, const ChunkList& list, CacheKind kind, cudaStream_t) {
  Launch& l = push(0, list);
  l.qa = a;
  l.kind = kind;
  return cudaSuccess;
}
cudaError_t launch_dequantise(const QuantArgs& a, const ChunkList& list, CacheKind kind, cudaStream_t) {
  Launch& l = push(1, list);
  l.qa = a;
  l.kind = kind;
  return cudaSuccess;
}
cudaError_t launch_chunk_rows(const ChunkArgs& a, const ChunkList& list, const ChunkUnits& units,
                              CacheKind kind, int rows, bool, cudaStream_t) {
  Launch& l = push(2, list);
  l.a = a;
  l.units = units;
  l.kind = kind;
  l.rows = rows;
  return cudaSuccess;
}
cudaError_t launch_chunk_tc(const ChunkArgs& a, const ChunkList& list, const ChunkUnits& units,
                            const DenseTiles& dense, const CUtensorMap&, CacheKind kind, bool,
                            cudaStream_t) {
  Launch& l = push(4, list);
  l.a = a;
  l.units = units;
  l.dense = dense;
  l.kind = kind;
  l.rows = a.rows_cta;
  return cudaSuccess;
}
cudaError_t launch_expand(const ChunkArgs& a, const ChunkList& list, const DenseTiles& dense,
                          CacheKind, cudaStream_t) {
  g_unfolds.push_back({static_cast<int>(g_launches.size()), list.n, a.dense, a.dense_rows, dense});
  return cudaSuccess;
}
cudaError_t launch_chunk_join(const ChunkArgs& a, const ChunkList& list, const ChunkUnits& units,
                              int rows, cudaStream_t) {
  Launch& l = push(3, list);
  l.a = a;
  l.units = units;
  l.rows = rows;
  return cudaSuccess;
}
}  // namespace td

// What cuTensorMapEncodeTiled checks, and that a box is 8 to 128 rows of 64.
static CUresult fake_encode(CUtensorMap*, CUtensorMapDataType, cuuint32_t rank, void* base,
                            const cuuint64_t* dims, const cuuint64_t* strides,
                            const cuuint32_t* box, const cuuint32_t*, CUtensorMapInterleave,
                            CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill) {
  const bool ok = rank == 2 && (reinterpret_cast<uintptr_t>(base) & 15) == 0 &&
                  strides[0] % 16 == 0 && strides[0] == dims[0] * 2 && dims[1] > 0 &&
                  dims[1] <= INT32_MAX && box[0] == 64 && box[1] >= 8 && box[1] <= 128 &&
                  box[1] % 8 == 0;
  return ok ? CUDA_SUCCESS : CUDA_ERROR_INVALID_VALUE;
}

extern "C" {

cudaError_t cudaGetDriverEntryPointByVersion(const char*, void** f, unsigned, unsigned long long,
                                             cudaDriverEntryPointQueryResult* q) {
  *f = reinterpret_cast<void*>(fake_encode);
  *q = cudaDriverEntryPointSuccess;
  return cudaSuccess;
}
cudaError_t cudaGetDevice(int* d) {
  *d = g_device;
  return cudaSuccess;
}
cudaError_t cudaMalloc(void** p, size_t bytes) {
  if (g_fail_malloc || bytes > g_room) return cudaErrorMemoryAllocation;
  g_floats = bytes / sizeof(float);
  // (an address of its own, 256-byte aligned, that nothing reads)
  static uintptr_t next = 0x100000000;
  *p = reinterpret_cast<void*>(next);
  next += (bytes + 255) / 256 * 256 + 256;
  g_held[*p] = bytes;
  return cudaSuccess;
}
cudaError_t cudaFree(void* p) {
  if (!g_synchronised || g_held.erase(p) != 1) return cudaErrorInvalidValue;
  g_synchronised = false;
  return cudaSuccess;
}
cudaError_t cudaStreamSynchronize(cudaStream_t) {
  g_synchronised = true;
  return g_fail_wait ? cudaErrorLaunchFailure : cudaSuccess;
}
cudaError_t cudaGetLastError(void) { return cudaSuccess; }
cudaError_t cudaStreamIsCapturing(cudaStream_t, cudaStreamCaptureStatus* s) {
  *s = g_capturing ? cudaStreamCaptureStatusActive : cudaStreamCaptureStatusNone;
  return cudaSuccess;
}

td_ctx* fake_ctx(const td_shape* s, int max_agents, int sms) {
  td_ctx* c = new td_ctx;
  c->shape = *s;
  c->g.H = s->n_kv_heads;
  c->g.D = s->head_dim;
  c->g.E = s->n_kv_heads * s->head_dim;
  c->g.half = s->head_dim / 2;
  c->max_agents = max_agents;
  c->device = 0;
  c->sm_count = sms;
  return c;
}
void fake_state(int device, int capturing, int fail_malloc) {
  g_device = device;
  g_capturing = capturing;
  g_fail_malloc = fail_malloc;
}
void fake_room(int64_t bytes) { g_room = static_cast<size_t>(bytes); }
void fake_reset(void) {
  g_launches.clear();
  g_unfolds.clear();
}
// Bytes that are held, of any context; buffers; whether waiting for a stream fails.
int64_t fake_held(void) {
  size_t sum = 0;
  for (const auto& h : g_held) sum += h.second;
  return static_cast<int64_t>(sum);
}
int fake_buffers(void) { return static_cast<int>(g_held.size()); }
void fake_wait(int fails) { g_fail_wait = fails != 0; }
int64_t fake_floats(void) { return static_cast<int64_t>(g_floats); }
int fake_launches(void) { return static_cast<int>(g_launches.size()); }
// what, kind, rows, n, direct, span, tok0, tokens, per_cta, lane_shift, head_mul, box_rows,
// whole_units, join_from
void fake_launch(int i, int64_t* out) {
  const Launch& l = g_launches[i];
  const bool quant = l.what < 2;
  const int64_t v[] = {l.what, l.kind, l.rows, l.list.n, l.a.direct, l.a.span,
                       quant ? l.qa.tok0 : 0, quant ? l.qa.tokens : l.a.tokens,
                       l.qa.per_cta, l.qa.lane_shift, l.qa.head_mul, l.a.box_rows, l.a.whole_units,
                       l.a.join_from};
  for (int k = 0; k < 14; ++k) out[k] = v[k];
}
int fake_unfolds(void) { return static_cast<int>(g_unfolds.size()); }
// The tiles' places of unfolding i; out: the attention launch that follows, its sequences, the
// copy's rows, whether that launch reads this copy with the same places, and where the scales
// and the partial results begin, in floats from the copy's begin.
void fake_unfold(int i, int32_t* base, int64_t* out) {
  const Unfold& u = g_unfolds[i];
  const Launch& l = g_launches[u.before];
  bool same = l.what == 4 && l.list.n == u.n && l.a.dense == u.to && l.a.dense_rows == u.rows;
  for (int x = 0; x <= u.n; ++x) {
    base[x] = u.dense.base[x];
    same = same && l.dense.base[x] == u.dense.base[x];
  }
  out[0] = u.before;
  out[1] = u.n;
  out[2] = u.rows;
  out[3] = same;
  out[4] = l.a.dense_scale - reinterpret_cast<const float*>(u.to);
  out[5] = l.a.part_o - reinterpret_cast<const float*>(u.to);
}
void fake_span(int start, int len, int window, int n_sink, int32_t* out) {
  const DenseSpan d = dense_span(start, len, window, n_sink);
  out[0] = d.s;
  out[1] = d.t0;
  out[2] = d.n;
}
void fake_list(int i, int32_t* agent, int32_t* start, int32_t* row, int32_t* base, int32_t* ns,
               int32_t* tok, int32_t* whole) {
  const Launch& l = g_launches[i];
  for (int x = 0; x <= l.list.n; ++x) {
    row[x] = l.list.row[x];
    base[x] = l.units.base[x];
    if (x < l.list.n) {
      agent[x] = l.list.agent[x];
      start[x] = l.list.start[x];
      ns[x] = l.units.nsplit[x];
      tok[x] = l.list.tok[x];
      whole[x] = l.units.whole[x];
    }
  }
}

}  // extern "C"
