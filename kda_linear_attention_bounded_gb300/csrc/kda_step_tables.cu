// Page tables and slot maps of one step over a paged cache, from the requests' lengths, in one launch.
//
// Request r has seq_lens[r] tokens in the cache and brings new_lens[r].  With exclusive sums over the requests
//   start_r = sum of new_lens,  taken_r = sum of grown,  grown_r = ceil((old + new) / page) - ceil(old / page)
// new token i of request r is row start_r + i at position old + i, new page j of request r is free_pages[taken_r + j]
// and goes to column ceil(old / page) + j of its table row, and a token's slot is page id * page + position % page.
//
// Bound by launch and load latency (the largest steps move a few MB).  Every CTA therefore scans the lengths itself,
// in windows of one request per thread, instead of waiting for a scan kernel: it then takes its share of the rows
// and of the new pages of the window, both found by binary search in the window's sums, so that one long prompt
// spreads over the grid as evenly as many short ones.  A token of a page handed out in this call reads the page id
// from the free list, never from the table, so no CTA waits for another's table writes.  The lengths in place (kv_lens is
// seq_lens) are one CTA's work: each is read once, by the thread that then writes it.
#include "kda_hybrid.cuh"

namespace kda {
namespace {

template <int kThreads>
__global__ void __launch_bounds__(kThreads) step_tables_kernel(StepTablesArgs p) {
  constexpr int kWarps = kThreads / 32;
  __shared__ int64_t s_start[kThreads + 1], s_taken[kThreads + 1];
  __shared__ int s_old[kThreads], s_had[kThreads];
  __shared__ bool s_refused[kThreads];
  __shared__ int64_t s_warp[2][kWarps];

  sm100::grid_dependency_wait();
  sm100::grid_launch_dependents();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t stride = static_cast<int64_t>(gridDim.x) * kThreads, mine = static_cast<int64_t>(blockIdx.x) * kThreads + tid;
  int64_t rows = 0, pages = 0, granted = 0;   // sums before the window; pages handed out
  for (int r0 = 0; r0 < p.B; r0 += kThreads) {
    const int r = r0 + tid;
    int64_t count = 0, grown = 0;
    int old = 0, had = 0;
    uint32_t bad = 0;
    if (r < p.B) {
      old = p.seq_lens[r];
      count = p.new_lens[r];
      if (old < 0 || count < 0 || old + count > INT32_MAX) {   // not lengths: nothing of the request is taken
        bad = KDA_DEVICE_BAD_COUNT;
        old = max(old, 0);
        count = 0;
      }
      had = static_cast<int>((static_cast<int64_t>(old) + p.page - 1) / p.page);
      const int64_t has = (old + count + p.page - 1) / p.page;
      grown = has - had;
      if (has > p.width) {          // its table row has no room
        bad |= KDA_DEVICE_NO_PAGES;
        grown = 0;
      }
    }
    // exclusive sums of (rows, pages) over the window
    int64_t a = count, b = grown;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t ua = __shfl_up_sync(0xffffffffu, a, o), ub = __shfl_up_sync(0xffffffffu, b, o);
      if (lane >= o) {
        a += ua;
        b += ub;
      }
    }
    __syncthreads();   // the last window's tables have been read
    if (lane == 31) {
      s_warp[0][warp] = a;
      s_warp[1][warp] = b;
    }
    __syncthreads();
    int64_t wa = 0, wb = 0, ta = 0, tb = 0;
#pragma unroll 8
    for (int w = 0; w < kWarps; ++w) {
      const int64_t xa = s_warp[0][w], xb = s_warp[1][w];
      if (w < warp) {
        wa += xa;
        wb += xb;
      }
      ta += xa;
      tb += xb;
    }
    const int64_t start = rows + wa + a - count, taken = pages + wb + b - grown;
    // Pages go out in request order, so once a request finds too few, so does every later one that needs any: places behind the
    // list, or of negative ids, which stand behind the others.
    const bool refused = (bad & KDA_DEVICE_NO_PAGES) ||
                         (grown > 0 && (taken + grown > p.num_free || p.free_pages[taken + grown - 1] < 0));
    s_start[tid] = start;
    s_taken[tid] = taken;
    s_old[tid] = old;
    s_had[tid] = had;
    s_refused[tid] = refused;
    if (tid == kThreads - 1) {
      s_start[kThreads] = rows + ta;
      s_taken[kThreads] = pages + tb;
    }
    if (r < p.B && blockIdx.x == (r0 / kThreads) % gridDim.x) {
      p.cu_seqlens[r + 1] = static_cast<int>(min(start + count, static_cast<int64_t>(INT32_MAX)));
      if (r == 0) p.cu_seqlens[0] = 0;
      p.kv_lens[r] = refused ? old : old + static_cast<int>(count);
      if (refused) bad |= KDA_DEVICE_NO_PAGES;
      if (start + count > p.max_tokens) bad |= KDA_DEVICE_BAD_COUNT;
      if (bad) atomicOr(p.status, bad);
    }
    __syncthreads();
    // new pages of the window, in the order of the free list
    const int64_t page_end = min(s_taken[kThreads], static_cast<int64_t>(p.num_free));
    for (int64_t j = s_taken[0] + mine; j < page_end; j += stride) {
      int lo = 0, hi = kThreads - 1;   // the last request with taken <= j
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (s_taken[mid] <= j) lo = mid; else hi = mid - 1;
      }
      if (!s_refused[lo])
        p.table[static_cast<int64_t>(r0 + lo) * p.table_stride + s_had[lo] + (j - s_taken[lo])] = p.free_pages[j];
    }
    // rows of the window
    const int64_t row_end = min(s_start[kThreads], p.max_tokens);
    for (int64_t t = s_start[0] + mine; t < row_end; t += stride) {
      int lo = 0, hi = kThreads - 1;   // the last request with start <= t
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (s_start[mid] <= t) lo = mid; else hi = mid - 1;
      }
      const int pos = s_old[lo] + static_cast<int>(t - s_start[lo]);
      const int col = pos / p.page, off = pos - col * p.page;
      int64_t slot = -1;
      if (!s_refused[lo]) {
        const int id = col < s_had[lo] ? p.table[static_cast<int64_t>(r0 + lo) * p.table_stride + col]
                                       : p.free_pages[s_taken[lo] + col - s_had[lo]];
        if (id >= 0) slot = static_cast<int64_t>(id) * p.page + off;
        else atomicOr(p.status, KDA_DEVICE_BAD_SLOT);
      }
      p.positions[t] = pos;
      p.slot_map[t] = slot;
    }
    // pages handed out so far: up to the first refusal for want of pages
    if (blockIdx.x == 0) {
      __shared__ unsigned long long s_granted;
      if (tid == 0) s_granted = 0;
      __syncthreads();
      if (!refused && grown > 0) atomicMax(&s_granted, static_cast<unsigned long long>(taken + grown));
      __syncthreads();
      granted = max(granted, static_cast<int64_t>(s_granted));
    }
    rows += ta;
    pages += tb;
  }
  if (mine == 0) {
    *p.pages_used = static_cast<int>(granted);
    if (p.B == 0) p.cu_seqlens[0] = 0;
  }
  // rows behind the last request: padding of a captured bucket
  for (int64_t t = min(rows, p.max_tokens) + mine; t < p.max_tokens; t += stride) {
    p.positions[t] = 0;
    p.slot_map[t] = -1;
  }
}

}  // namespace

cudaError_t launch_step_tables(const StepTablesArgs &a, cudaStream_t stream) {
  // a window holds the whole batch where it can (512 requests: 6.0 us with 512 threads, 7.8 with 1024)
  const int threads = a.B <= 256 ? 256 : a.B <= 512 ? 512 : 1024;
  const int64_t want = (a.max_tokens + threads - 1) / threads;
  const unsigned grid = static_cast<unsigned>(want < 1 || a.one_cta ? 1 : want > 608 ? 608 : want);
  const auto kernel = threads == 256 ? step_tables_kernel<256> : threads == 512 ? step_tables_kernel<512> : step_tables_kernel<1024>;
  return launch_dependent(kernel, grid, threads, 0, stream, a);
}

}  // namespace kda
