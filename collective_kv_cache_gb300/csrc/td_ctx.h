// td_ctx.h - the context behind include/td.h's td_ctx and the host helpers its entry points
// share (td_host.cpp, td_chunks.cpp).
#pragma once

#include <cuda_runtime.h>

#include <cstdint>
#include <new>
#include <vector>

#include "td.h"
#include "td_internal.h"

namespace td {

// A context's buffer that grows with its calls.
struct Scratch {
  float* p = nullptr;
  size_t cap = 0;                   // its size in floats
  bool kept = false;                // a captured call has used it
};

}  // namespace td

struct td_ctx {
  td_shape shape;
  td::Geom g;
  int max_agents, max_blocks, max_shared, max_nb, nbw_max;
  int device;

  // round tables (device) and their pinned staging
  int32_t* d_off = nullptr;
  float* d_cos = nullptr;
  float* d_sin = nullptr;
  int32_t* d_tok_block = nullptr;
  int32_t* d_blk_start = nullptr;
  unsigned char* h_stage = nullptr;
  size_t stage_bytes = 0;
  cudaEvent_t stage_done = nullptr;
  bool stage_pending = false;

  // Streams that have read the round tables since their last upload, each with an event
  // recorded after its latest launch. A round change makes the uploading stream wait on
  // all of them; a stream's first call after an upload waits on tables_ready.
  struct StreamUse {
    cudaStream_t stream;
    cudaEvent_t last_use;
    bool ordered;      // ordered after the current tables' upload
  };
  std::vector<StreamUse> users;
  cudaEvent_t tables_ready = nullptr;
  cudaStream_t tables_stream = nullptr;
  bool tables_recorded = false;

  // cached round (host copy) and its device view
  bool have_round = false;
  int N = 0, M = 0, S = 0;
  std::vector<int32_t> c_len, c_hist, c_perm;

  // scratch
  float* d_dev = nullptr;           // [max_agents * max_shared]
  int32_t* d_pos = nullptr;         // [max_agents * max_shared] prompt position of each token
  uint32_t* d_sel_hist = nullptr;   // [max_agents * kSelHistBins] selection histograms (zero)
  float* d_gdev = nullptr;          // [max_shared] group deviation (variant)
  double* d_score = nullptr;        // [max_agents] deviation totals (variant)
  uint32_t* d_selbits = nullptr;    // [max_agents * max_nb]
  int32_t* d_firstrank = nullptr;   // [max_agents * max_nb]
  uint32_t* d_mask = nullptr;       // [max_agents * nbw_max]
  uint32_t* d_cand = nullptr;       // [max_agents * nbw_max]
  uint32_t* d_pm_mask = nullptr;    // [max_agents * nbw_max] masks of td_pick_master
  int32_t* d_wprefix = nullptr;     // [max_agents * nbw_max + max_agents]
  int64_t* d_aprefix = nullptr;     // [max_agents + 1]
  uint32_t* d_flag = nullptr;       // [max_agents * L * max_nb] flags + [max_agents * L] counts
  int sm_count = 0;                 // of the context's device
  int32_t* d_ints = nullptr;        // encode's words (unused, m_ok, over, prep_done), spare,
                                    // pick_master's counter, spare
  int64_t* d_bound = nullptr;
  uint32_t* d_err = nullptr;
  td::Scratch attn;                 // attention partials
  uint32_t attn_tx_pad = 0;         // fault injection: bytes the attention never receives
  td::Scratch chunk;                // chunk attention's unfolded pages and partial results
  uint32_t chunk_launched = 0;      // its kernels that this context has launched, a bit each
  std::vector<float*> outgrown;     // scratch that captured calls have used, and that was too small
  // pinned host words for results
  int64_t* h_words = nullptr;       // [4]
};

namespace td {

inline bool is_pow2(int x) { return x > 0 && (x & (x - 1)) == 0; }
inline int log2i(int x) {
  int s = 0;
  while ((1 << s) < x) ++s;
  return s;
}

inline bool same_device(const td_ctx* c) {
  int d = -1;
  return cudaGetDevice(&d) == cudaSuccess && d == c->device;
}

inline bool capturing(cudaStream_t st) {
  cudaStreamCaptureStatus cs = cudaStreamCaptureStatusNone;
  if (cudaStreamIsCapturing(st, &cs) != cudaSuccess) {
    cudaGetLastError();
    return false;
  }
  return cs != cudaStreamCaptureStatusNone;
}

// Scratch of at least `need` floats, `more` of them where that is to be had. A buffer that a
// captured call has used stays until the context goes, since the graph holds its address; any
// other is freed when it is outgrown, after the stream's work (the context's earlier calls of
// the group are ordered before this one). Inside a capture nothing can be allocated.
inline td_status grow(td_ctx* c, Scratch* s, size_t need, size_t more, cudaStream_t st) {
  if (need == 0) return TD_OK;
  const bool captured = capturing(st);
  if (need <= s->cap) {
    s->kept |= captured;
    return TD_OK;
  }
  if (captured) return TD_ERR_INVALID_ARG;
  if (s->p && s->kept) {
    try {
      c->outgrown.reserve(c->outgrown.size() + 1);
    } catch (const std::bad_alloc&) {
      return TD_ERR_CUDA;
    }
  } else if (s->p) {
    if (cudaStreamSynchronize(st) != cudaSuccess || cudaFree(s->p) != cudaSuccess) {
      cudaGetLastError();
      return TD_ERR_CUDA;
    }
    *s = Scratch{};
  }
  float* p = nullptr;
  size_t cap = more > need ? more : need;
  if (cudaMalloc(&p, cap * sizeof(float)) != cudaSuccess) {
    cudaGetLastError();
    cap = need;
    if (cudaMalloc(&p, cap * sizeof(float)) != cudaSuccess) {
      cudaGetLastError();
      return TD_ERR_CUDA;
    }
  }
  if (s->p) c->outgrown.push_back(s->p);
  *s = Scratch{p, cap, false};
  return TD_OK;
}

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// cuTensorMapEncodeTiled from the driver, looked up once (no link-time dependency).
typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                  const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                  const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

inline EncodeTiledFn encode_tiled() {
  static EncodeTiledFn fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q = cudaDriverEntryPointSymbolNotFound;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                         &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      return static_cast<EncodeTiledFn>(nullptr);
    return reinterpret_cast<EncodeTiledFn>(p);
  }();
  return fn;
}

}  // namespace td
