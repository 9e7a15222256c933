// k_tables.cu - block tables and slot maps from the requests' lengths.
//
// Request x goes from len to len + add positions, so from ceil(len / P) pages to ceil((len + add)
// / P). With prefix sums over the requests of the tokens t, the pages taken a and the pages given
// back f, everything else is a function of its place alone: the j-th page taken in all is the
// j-th one given back while there are such (they go on top of the list, the first request's first
// page uppermost) and then pages[count - 1 - (j - f)] of the list; the i-th page given back that
// nobody takes goes to pages[count + f - 1 - i].
//
// It reads three words a request and writes one a token: a few microseconds, bound by the launch
// and the latency of the sums, not by memory (4.4 us a call of 64 requests in a graph; 256 prompts of
// 553,000 tokens mapped and given back 11 us, with a group of lanes a page and 64-bit sums 18). So it
// is one launch: every CTA takes the sums over all requests itself (at most 4096, from L2) instead of
// waiting for another kernel, then its share of the pages: a thread finds a page that new tokens
// touch, its warp writes the slots of its 32, and a thread takes a page that goes back on the list. An
// entry is read and written by the one thread that has its page, so nothing needs an order among CTAs
// but the lengths and the count, which every CTA reads: the last one to finish, told by a ticket,
// writes those.
#include "td_device.cuh"

namespace td {

namespace {

constexpr int kThreads = kTablesThreads;
constexpr int kWarpsT = kThreads / 32;

// Sums over requests, none past kMany: a sum of numbers that are not negative stays there once it is
// there, whichever are added first, and a call that reaches it is refused.
constexpr uint32_t kMany = INT32_MAX;

struct Sums {
  uint32_t items, tokens, taken, given;
  __device__ __forceinline__ void add(const Sums& o) {
    items = min(items + o.items, kMany);
    tokens = min(tokens + o.tokens, kMany);
    taken = min(taken + o.taken, kMany);
    given = min(given + o.given, kMany);
  }
};

__device__ __forceinline__ uint32_t up(uint32_t v, int o) {
  return __shfl_up_sync(0xFFFFFFFFu, v, o);
}

// The last x with first[x] <= i (first[0] = 0; i below the array's end value).
__device__ __forceinline__ int find(const int32_t* first, int n, int i) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (first[mid] <= i) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

}  // namespace

__global__ void __launch_bounds__(kThreads) tables_kernel(const __grid_constant__ TablesArgs A) {
  extern __shared__ int32_t s_dyn[];
  const int n = A.n, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int32_t* s_item = s_dyn;                 // pages that new tokens touch, before request x
  int32_t* s_tok = s_item + n + 1;         // new tokens
  int32_t* s_take = s_tok + n + 1;         // pages taken
  int32_t* s_give = s_take + n + 1;        // pages given back
  uint32_t* s_seen = reinterpret_cast<uint32_t*>(s_give + n + 1);    // rows named
  __shared__ Sums s_warp[kWarpsT];
  __shared__ int s_last;
  pdl_wait();
  const int P = A.P;
  const int per = (n + kThreads - 1) / kThreads, x0 = min(n, tid * per), x1 = min(n, x0 + per);
  // a request: its lengths before and after, its row
  struct Request {
    int len;
    int64_t end;
    int row;
  };
  auto request = [&](int x) {
    const int len = A.len[x];
    return Request{len, static_cast<int64_t>(len) + A.add[x], A.row ? A.row[x] : x};
  };
  const int count = *A.count;
  Request first{0, 0, 0};                  // (on its way while the bits are cleared)
  if (x0 < x1) first = request(x0);
  for (int i = tid; i < (A.max_rows + 31) / 32; i += kThreads) s_seen[i] = 0u;
  __syncthreads();
  const int64_t most = min(static_cast<int64_t>(A.max_lp) * P, static_cast<int64_t>(INT32_MAX / 2));
  bool bad = count < 0 || count > A.capacity, full = false;
  auto check = [&](const Request& q) {
    if (q.row < 0 || q.row >= A.max_rows) bad = true;
    else if ((atomicOr(s_seen + (q.row >> 5), 1u << (q.row & 31)) >> (q.row & 31)) & 1u) bad = true;
    if (q.len < 0 || q.end < 0) bad = true;
    else if (max(static_cast<int64_t>(q.len), q.end) > most) full = true;
  };
  // (of a request that is refused any numbers do)
  auto sums_of = [&](const Request& q) {
    Sums s{0u, 0u, 0u, 0u};
    const uint32_t len = static_cast<uint32_t>(q.len) & kMany, end = static_cast<uint32_t>(q.end) & kMany;
    const uint32_t p = static_cast<uint32_t>(P), have = (len + p - 1) / p, want = (end + p - 1) / p;
    if (end > len) {
      s.items = want - len / p;
      s.tokens = end - len;
      s.taken = want - have;
    } else {
      s.given = have - want;
    }
    return s;
  };
  Sums mine{0u, 0u, 0u, 0u};
  for (int x = x0; x < x1; ++x) {
    const Request q = x == x0 ? first : request(x);
    check(q);
    mine.add(sums_of(q));
  }
  Sums before = mine;                      // inclusive over the warp, then exclusive over the CTA
#pragma unroll
  for (int o = 1; o < 32; o *= 2) {
    const Sums v{up(before.items, o), up(before.tokens, o), up(before.taken, o), up(before.given, o)};
    if (lane >= o) before.add(v);
  }
  if (lane == 31) s_warp[warp] = before;
  bad = __syncthreads_or(bad);
  full = __syncthreads_or(full);
  // (as the sums have not reached kMany)
  before.items -= mine.items;
  before.tokens -= mine.tokens;
  before.taken -= mine.taken;
  before.given -= mine.given;
  Sums all{0u, 0u, 0u, 0u};
#pragma unroll
  for (int w = 0; w < kWarpsT; ++w) {
    if (w < warp) before.add(s_warp[w]);
    all.add(s_warp[w]);
  }
  const int64_t left = static_cast<int64_t>(count) + all.given - all.taken;
  full = full || all.tokens > static_cast<uint32_t>(A.max_slots) || left < 0 || left > A.capacity ||
         max(max(all.items, all.tokens), max(all.taken, all.given)) >= kMany;
  const bool ok = !bad && !full;
  const TablesIndex gthread = blockIdx.x * kThreads + tid, gthreads = gridDim.x * kThreads;
  const TablesIndex max_slots = static_cast<TablesIndex>(A.max_slots);
  if (!ok) {
    if (gthread == 0) atomicOr(A.err, err_bit(bad ? TD_ERR_INVALID_ARG : TD_ERR_CAPACITY));
    if (A.token_start && blockIdx.x == 0)
      for (int x = tid; x <= n; x += kThreads) A.token_start[x] = 0;
    for (TablesIndex i = gthread; i < max_slots; i += gthreads) A.slots[i] = -1;
    pdl_trigger();
    return;
  }
  for (int x = x0; x < x1; ++x) {
    s_item[x] = static_cast<int32_t>(before.items);
    s_tok[x] = static_cast<int32_t>(before.tokens);
    s_take[x] = static_cast<int32_t>(before.taken);
    s_give[x] = static_cast<int32_t>(before.given);
    if (x + 1 < x1) before.add(sums_of(x == x0 ? first : request(x)));
  }
  if (tid == 0) s_tok[n] = static_cast<int32_t>(all.tokens);
  __syncthreads();
  pdl_trigger();
  const TablesIndex items = all.items, taken = all.taken, tokens = all.tokens;
  const int given = static_cast<int>(all.given);
  auto entry = [&](int x, int lp) {
    return A.bt + static_cast<int64_t>(A.row ? A.row[x] : x) * A.max_lp + lp;
  };
  // the place in the table of the i-th page given back
  auto returned = [&](int i) {
    const int x = find(s_give, n, i);
    const int end = A.len[x] + A.add[x];
    return entry(x, pages_of(end, P) + i - s_give[x]);
  };
  int gs = 1;                              // lanes that write a page's slots
  while (gs < P && gs < 32) gs *= 2;
  const int sub = lane & (gs - 1), group = lane / gs;
  bool hole = false;
  // a lane finds a page, then the warp writes the slots of its 32
  for (TablesIndex i0 = gthread - lane; i0 < items; i0 += gthreads) {
    int page = -1, lo = 0, hi = 0, to_slot = 0;       // its new tokens [lo, hi), and slot 0's place
    if (i0 + lane < items) {
      const int i = static_cast<int>(i0 + lane), x = find(s_item, n, i);
      const int len = A.len[x], end = len + A.add[x];
      const int lp = len / P + i - s_item[x], have = pages_of(len, P);
      int32_t* to = entry(x, lp);
      if (lp < have) {
        page = *to;
      } else {
        const int j = s_take[x] + lp - have;
        if (j < given) {
          int32_t* from = returned(j);
          page = *from;
          *from = -1;
        } else {
          page = A.pages[count - 1 - (j - given)];
        }
      }
      if (page < 0 || page >= A.num_pages) {
        page = -1;
        hole = true;
      }
      if (lp >= have) *to = page;
      lo = max(len - lp * P, 0);
      hi = min(end - lp * P, P);
      to_slot = s_tok[x] + (lp * P - len);
    }
    const int most_here = static_cast<int>(min(32u, items - i0));
    for (int k = group; k - group < most_here; k += 32 / gs) {       // (as many rounds for every lane)
      const int k_page = __shfl_sync(0xFFFFFFFFu, page, k), k_to = __shfl_sync(0xFFFFFFFFu, to_slot, k);
      const int k_lo = __shfl_sync(0xFFFFFFFFu, lo, k), k_hi = __shfl_sync(0xFFFFFFFFu, hi, k);
      for (int s = sub; s < k_hi; s += gs)
        if (s >= k_lo) A.slots[k_to + s] = k_page < 0 ? -1 : k_page * P + s;
    }
  }
  for (TablesIndex i = taken + gthread; i < all.given; i += gthreads) {
    int32_t* from = returned(static_cast<int>(i));
    const int page = *from;
    hole |= page < 0 || page >= A.num_pages;
    A.pages[count + (given - 1 - static_cast<int>(i))] = page;
    *from = -1;
  }
  if (hole) atomicOr(A.err, err_bit(TD_ERR_UNMAPPED_PAGE));
  if (A.token_start && blockIdx.x == 0)
    for (int x = tid; x <= n; x += kThreads) A.token_start[x] = s_tok[x];
  for (TablesIndex i = tokens + gthread; i < max_slots; i += gthreads) A.slots[i] = -1;
  // every CTA has read the lengths and the count: the last one replaces them
  __syncthreads();
  if (tid == 0) {
    __threadfence();
    s_last = atomicAdd(A.ticket, 1) == static_cast<int>(gridDim.x) - 1;
    if (s_last) *A.ticket = 0;
  }
  __syncthreads();
  if (!s_last) return;
  for (int x = tid; x < n; x += kThreads) A.len[x] += A.add[x];
  if (tid == 0) *A.count = static_cast<int32_t>(left);
}

// Dynamic shared memory for n requests of a table of max_rows rows.
static constexpr size_t tables_smem(int n, int max_rows) {
  return (static_cast<size_t>(n + 1) * 4 + (max_rows + 31) / 32) * 4;
}

cudaError_t launch_tables(const TablesArgs& a, int sm_count, cudaStream_t st) {
  const unsigned grid = tables_grid(a, sm_count);
  const size_t smem = tables_smem(a.n, a.max_rows);
  // (what a block may have unasked covers the static part too; what is asked for holds for the device,
  // whoever calls, so it is the same for every call)
  if (smem > 47 * 1024) {
    const cudaError_t e =
        cudaFuncSetAttribute(tables_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(tables_smem(kMaxAgents, kMaxAgents)));
    if (e != cudaSuccess) return e;
  }
  return launch_after(tables_kernel, grid, kThreads, smem, st, a);
}

}  // namespace td
