// The pages' own operations: requests forked and ended, the cache compacted, pages copied.  Pages in use are those that the
// table's rows hold in their first ceil(length / page) places; nothing is counted from call to call.
//
// Forking.  Fork i needs a page where its parent's length n is no multiple of the page, and takes the free list's entry at the
// number of forks before it that need one.  Every CTA counts them for itself, in windows of a fork a thread, and then copies the
// rows of its own forks.  The list ends with its length or at its first negative id: each thread reads its own fork's entry, and
// the least place of a negative one is the end for this window and those behind it.  Bound by latency: lengths, counts, ids, rows.
//
// Ending and compacting.  One cluster of CTAs has a bit for each page in each of its CTAs' shared memory (in windows of the ids
// where there are more).  Its warps take the rows in pieces of 256 places and set the bits of what they hold, each in its own
// CTA's bits (where a prompt's pages are held by many rows, most find their bit set).  Then each CTA joins an equal part of the
// words through the cluster, every CTA fetches all parts and sums the bits before each word, and writes its part of the lists:
// places in a list are such sums, so the lists are in ascending order whatever came first.  With n pages in use, the i-th one of id
// n or above goes to the i-th free id below n; a place of the table finds its number by the same sums (in windows: in the list).
// Bound by latency: lengths, ids, three meetings of the cluster.
// Large tables are marked by all SMs instead, with atomics on bits in the free list's own memory, which is written over once all have
// read them; where requests end, all SMs write the list, too.  Bound by the latency of four launches in a row, and by the atomics.
//
// Copying.  Bound by HBM.  Every CTA lists the pairs of a window that are copies; pieces of 8 KB of them all stand in one line, of
// which each warp takes every so-manieth.  (Read and written, of 0.5 GB: pages of 1 MB 6170 GB/s, of 8 KB 5550, of 12 KB, whose last
// pieces are a plain loop's, 4860, of 4 KB 4370.)  A list is gone through by every CTA, what is no copy, too: ten copies in one of
// 100000 entries take 182 us, in one of 450000 827.
#include <algorithm>
#include <type_traits>

#include "kda_cache.h"
#include "kda_hybrid.cuh"

namespace kda {
namespace {

// Pages that a row holds; a length that is none, or that the row has no room for, counts as 0.
__device__ __forceinline__ int pages_of(const TableArgs &t, int len, bool record) {
  const int pages = len > 0 ? (len - 1) / t.page + 1 : 0;
  if (len < 0 || pages > t.width) {
    if (record) atomicOr(t.status, KDA_DEVICE_BAD_COUNT);
    return 0;
  }
  return pages;
}

__device__ __forceinline__ int warp_scan(int x, int lane) {   // inclusive
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += u;
  }
  return x;
}

// ---------------------------------------------------------------- forking
constexpr int kForkThreads = 256;
__global__ void __launch_bounds__(kForkThreads) fork_requests_kernel(ForkArgs p) {
  constexpr int kWarps = kForkThreads / 32;
  __shared__ int s_len[kForkThreads], s_parent[kForkThreads], s_child[kForkThreads], s_taken[kForkThreads], s_page[kForkThreads];
  __shared__ int s_warp[kWarps], s_end;
  sm100::grid_dependency_wait();
  sm100::grid_launch_dependents();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int before = 0;   // pages that the forks before the window need
  if (tid == 0) s_end = p.num_free;   // the first place behind the list's ids, as far as it has been read
  for (int f0 = 0; f0 < p.forks; f0 += kForkThreads) {
    const int f = f0 + tid;
    int parent = -1, child = -1, len = 0, need = 0;
    uint32_t bad = 0;
    if (f < p.forks) {
      parent = p.parents[f];
      child = p.children[f];
      if (parent < 0 || child < 0) {
        child = -1;
      } else if (parent >= p.t.B || child >= p.t.B || parent == child) {
        bad = KDA_DEVICE_BAD_INDEX;
        child = -1;
      } else {
        len = p.seq_lens[parent];
        if (len < 0 || (len > 0 && (len - 1) / p.t.page >= p.t.width)) {
          bad = KDA_DEVICE_BAD_COUNT;
          child = -1;
        } else {
          need = len % p.t.page != 0;
        }
      }
    }
    const uint32_t on = __ballot_sync(0xffffffffu, need);
    __syncthreads();   // the last window's lists have been read
    if (lane == 0) s_warp[warp] = __popc(on);
    __syncthreads();
    int taken = before + __popc(on & ((1u << lane) - 1));   // (below the number of forks)
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) taken += s_warp[w];
      before += s_warp[w];
    }
    const int page = need && taken < s_end ? p.free_pages[taken] : -1;
    if (need && page < 0) atomicMin(&s_end, taken);
    s_len[tid] = len;
    s_parent[tid] = parent;
    s_child[tid] = child;
    s_taken[tid] = need ? taken : -1;
    s_page[tid] = page;
    __syncthreads();
    const int end = s_end;
    if (need && taken >= end) bad |= KDA_DEVICE_NO_PAGES;
    if (bad && blockIdx.x == 0) atomicOr(p.t.status, bad);
    for (int j = (blockIdx.x + gridDim.x - f0 % gridDim.x) % gridDim.x; j < kForkThreads && f0 + j < p.forks; j += gridDim.x) {
      const int c = s_child[j], n = s_len[j], at = s_taken[j];
      if (c < 0 || at >= end) {
        if (tid == 0) p.copy_src[f0 + j] = p.copy_dst[f0 + j] = -1;
        continue;
      }
      const int32_t *from = p.t.table + s_parent[j] * p.t.stride;
      int32_t *to = p.table + c * p.t.stride;
      const int whole = n / p.t.page;
      for (int e = tid; e < whole; e += kForkThreads) to[e] = from[e];
      if (tid == 0) {
        int src = -1, dst = -1;
        if (at >= 0) {
          src = from[whole];
          dst = s_page[j];
          to[whole] = dst;
          if (src < 0) atomicOr(p.t.status, KDA_DEVICE_BAD_PAGE);   // (no copy is made)
        }
        p.copy_src[f0 + j] = src;
        p.copy_dst[f0 + j] = dst;
        p.seq_lens[c] = n;
      }
    }
  }
  __syncthreads();   // (without forks the end has just been set)
  if (blockIdx.x == 0 && tid == 0) *p.pages_used = min(before, s_end);
}

// ---------------------------------------------------------------- pages in use
constexpr int kThreads = 1024, kWarps = kThreads / 32;
constexpr int kMostRanks = 16;              // CTAs of the cluster
constexpr int kMostWords = 28 * 1024;       // words of bits: windows of 896 K ids (224 KB with their sums)
constexpr int kPiece = 256;                 // places of a row that a warp takes: 8 loads a lane, all under way together

__device__ __forceinline__ void cluster_sync() {
  __syncthreads();   // (whole warps come to the cluster's barrier)
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
// Four words of the shared memory of the cluster's CTA `rank`, at this CTA's address of them.
__device__ __forceinline__ uint4 peer_words(const uint32_t *p, uint32_t rank) {
  uint32_t at;
  uint4 v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(sm100::smem_u32(p)), "r"(rank));
  asm volatile("ld.shared::cluster.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at) : "memory");
  return v;
}

// The table's pieces in turn, by the warps of so many CTAs: f(row, first place, places, the lane's ids; none of a bad length).
template <typename F>
__device__ __forceinline__ void pieces_of(const TableArgs &t, const int32_t *seq_lens, uint32_t rank, int ranks, bool record, F f) {
  const int lane = threadIdx.x & 31;
  const int per_row = max(1, (t.width + kPiece - 1) / kPiece);
  const int64_t units = static_cast<int64_t>(per_row) * t.B;
  int64_t u = static_cast<int>(threadIdx.x >> 5) * ranks + static_cast<int>(rank);   // (few pieces go to all CTAs)
  const auto row_of = [&](int64_t x, int &piece) {
    piece = units >> 31 ? static_cast<int>(x / t.B) : static_cast<int>(static_cast<uint32_t>(x) / static_cast<uint32_t>(t.B));
    // (a long row's pieces go to different warps: each round of pieces begins some rows later)
    return static_cast<int>((x - static_cast<int64_t>(piece) * t.B + 37ll * piece) % t.B);
  };
  int piece = 0, b = 0, len = 0;
  if (u < units) {
    b = row_of(u, piece);
    len = __ldcg(seq_lens + b);
  }
  while (u < units) {
    const int pages = pages_of(t, len, record && piece == 0 && lane == 0), first = piece * kPiece, n = min(kPiece, pages - first), row = b;
    u += ranks * kWarps;
    if (u < units) {   // (the next one's length comes beside this one's ids)
      b = row_of(u, piece);
      len = __ldcg(seq_lens + b);
    }
    if (n <= 0) continue;
    const int32_t *from = t.table + row * t.stride + first;
    int id[kPiece / 32];
#pragma unroll
    for (int i = 0; i < kPiece / 32; ++i) id[i] = 32 * i + lane < n ? from[32 * i + lane] : 0;
    f(row, first, n, id);
  }
}

__device__ __forceinline__ void end_request(int32_t *seq_lens, int row, int B, uint32_t *status) {
  if (row >= B) atomicOr(status, KDA_DEVICE_BAD_INDEX);
  else if (row >= 0) seq_lens[row] = 0;
}

// The pages in use among the ids of a window: for every word of 32 its bits and how many bits are set before it.  Bits behind the
// window's last id are clear.
struct Window {
  uint32_t *own, *bits;   // what this CTA's warps found; the cluster's
  uint32_t *before;       // (in the place of own, which is done with by then)
  int from, words, span;
  int w0, w1;             // the words whose lists this CTA writes
  int set;                // bits set in all
};
__device__ __forceinline__ Window window_of(int num_pages, int from, int most, uint32_t *smem, uint32_t rank, int *per) {
  const int ranks = cluster_size();
  Window x;
  x.own = smem;
  x.bits = smem + most;
  x.before = smem;
  x.from = from;
  x.span = min(32 * most, num_pages - from);
  x.words = (x.span + 31) / 32;
  *per = (x.words + 4 * ranks - 1) / (4 * ranks) * 4;   // (16 bytes at a time)
  x.w0 = min(x.words, static_cast<int>(rank) * *per);
  x.w1 = min(x.words, x.w0 + *per);
  return x;
}
// The sums, with the bits there.
__device__ __forceinline__ void sum_bits(Window &x, uint32_t *s_warp) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  // (consecutive words a thread)
  const int chunk = (x.words + 4 * kThreads - 1) / (4 * kThreads) * 4, c0 = min(x.words, tid * chunk), c1 = min(x.words, c0 + chunk);
  int n = 0;
  for (int i = c0; i < c1; i += 4) {   // (words behind the last of them are clear)
    const uint4 y = *reinterpret_cast<const uint4 *>(x.bits + i);
    n += __popc(y.x) + __popc(y.y) + __popc(y.z) + __popc(y.w);
  }
  const int inc = warp_scan(n, lane);
  if (lane == 31) s_warp[warp] = inc;
  __syncthreads();
  const int of_warp = s_warp[lane], up_to = warp_scan(of_warp, lane);   // (as many warps as lanes)
  x.set = __shfl_sync(0xffffffffu, up_to, 31);
  int sum = inc - n + __shfl_sync(0xffffffffu, up_to - of_warp, warp);
  for (int i = c0; i < c1; i += 4) {
    const uint4 y = *reinterpret_cast<const uint4 *>(x.bits + i);
    const int a = sum + __popc(y.x), b = a + __popc(y.y), c = b + __popc(y.z);
    *reinterpret_cast<int4 *>(x.before + i) = make_int4(sum, a, b, c);
    sum = c + __popc(y.w);
  }
  __syncthreads();
}
__device__ __forceinline__ Window mark(const TableArgs &t, const int32_t *seq_lens, int num_pages, int from, int most, uint32_t *smem,
                                       uint32_t *s_warp, uint32_t rank, bool record) {
  const int tid = threadIdx.x, ranks = cluster_size();
  int per;
  Window x = window_of(num_pages, from, most, smem, rank, &per);
  const int lane = tid & 31;
  for (int i = tid; i < ((x.words + 3) & ~3); i += kThreads) x.own[i] = 0;
  __syncthreads();
  pieces_of(t, seq_lens, rank, ranks, record, [&](int, int, int n, const int (&id)[kPiece / 32]) {
    bool bad = false;
    uint32_t at[kPiece / 32], old[kPiece / 32];
#pragma unroll
    for (int i = 0; i < kPiece / 32; ++i) {   // (words that are set meanwhile are set again)
      const bool there = 32 * i + lane < n;
      bad |= there && (id[i] < 0 || id[i] >= num_pages);
      at[i] = static_cast<uint32_t>(id[i]) - static_cast<uint32_t>(from);
      if (!there || id[i] < from || at[i] >= static_cast<uint32_t>(x.span)) at[i] = ~0u;
      old[i] = at[i] == ~0u ? ~0u : x.own[at[i] >> 5];
    }
#pragma unroll
    for (int i = 0; i < kPiece / 32; ++i) {
      const uint32_t bit = 1u << (at[i] & 31);
      if (!(old[i] & bit)) atomicOr(x.own + (at[i] >> 5), bit);
    }
    if (record && bad) atomicOr(t.status, KDA_DEVICE_BAD_PAGE);
  });
  cluster_sync();
  // an equal part of the words joined by each CTA, then all parts to all
  for (int i = x.w0 + 4 * tid; i < x.w1; i += 4 * kThreads) {
    uint4 y = make_uint4(0, 0, 0, 0);
#pragma unroll
    for (uint32_t r = 0; r < kMostRanks; ++r) {
      const uint4 z = peer_words(x.own + i, min(r, static_cast<uint32_t>(ranks) - 1));   // (all under way together)
      y.x |= z.x; y.y |= z.y; y.z |= z.z; y.w |= z.w;
    }
    *reinterpret_cast<uint4 *>(x.bits + i) = y;
  }
  cluster_sync();
#pragma unroll 4
  for (int i = 4 * tid; i < x.words; i += 4 * kThreads)
    if (i < x.w0 || i >= x.w1) *reinterpret_cast<uint4 *>(x.bits + i) = peer_words(x.bits + i, static_cast<uint32_t>(i / per));
  __syncthreads();
  sum_bits(x, s_warp);
  return x;
}

// ---- tables of many places: marked by the whole GPU, in words where the free list will be
__global__ void __launch_bounds__(256) clear_marks_kernel(uint32_t *words, int count, int32_t *seq_lens, const int32_t *rows, int num_rows, int B,
                                                          uint32_t *status) {
  sm100::grid_dependency_wait();
  sm100::grid_launch_dependents();
  const int tid = blockIdx.x * 256 + threadIdx.x, threads = gridDim.x * 256;
  for (int i = 4 * tid; i < count; i += 4 * threads) *reinterpret_cast<uint4 *>(words + i) = make_uint4(0, 0, 0, 0);
  for (int i = tid; i < num_rows; i += threads) end_request(seq_lens, rows[i], B, status);
}
__global__ void __launch_bounds__(kThreads, 1) mark_pages_kernel(TableArgs t, const int32_t *seq_lens, int num_pages, uint32_t *words) {
  sm100::grid_dependency_wait();
  sm100::grid_launch_dependents();
  const int lane = threadIdx.x & 31;
  pieces_of(t, seq_lens, blockIdx.x, gridDim.x, true, [&](int, int, int n, const int (&id)[kPiece / 32]) {
    bool bad = false;
#pragma unroll
    for (int i = 0; i < kPiece / 32; ++i) {
      const bool there = 32 * i + lane < n, on = there && id[i] >= 0 && id[i] < num_pages;
      bad |= there && !on;
      const int w = on ? id[i] >> 5 : -1;
      uint32_t bit = on ? 1u << (id[i] & 31) : 0u;
      // Ids in a row have few words: one lane sets what the first lane's and the last lane's words get.  (512 rows of one prompt with such ids:
      // 376 us without.)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const bool same = w == __shfl_sync(0xffffffffu, w, 31 * k);
        if (__popc(__ballot_sync(0xffffffffu, same && bit)) < 2) continue;
        const uint32_t bits = __reduce_or_sync(0xffffffffu, same ? bit : 0u);
        if (same) bit = 0;
        if (lane == 31 * k) bit = bits;   // (after its own word's round a lane has no bit but what it sets for all)
      }
      if (bit) atomicOr(words + w, bit);
    }
    if (bad) atomicOr(t.status, KDA_DEVICE_BAD_PAGE);
  });
}
// The window of all ids from such words.  Behind it they may be written over.
__device__ __forceinline__ Window marked(const uint32_t *words, int num_pages, int most, uint32_t *smem, uint32_t *s_warp, uint32_t rank) {
  int per;
  Window x = window_of(num_pages, 0, most, smem, rank, &per);
#pragma unroll 4
  for (int i = 4 * threadIdx.x; i < x.words; i += 4 * kThreads)
    *reinterpret_cast<uint4 *>(x.bits + i) = __ldcg(reinterpret_cast<const uint4 *>(words + i));
  cluster_sync();
  sum_bits(x, s_warp);
  return x;
}

// Ids of this CTA's words that `pick(word's place)` has bits for, to out[place(word's place)] on, from out[begin] on: a warp writes a
// word's ids.
template <typename P, typename O>
__device__ __forceinline__ void write_ids(const Window &x, int32_t *out, P pick, O place, int begin = 0) {
  const int lane = threadIdx.x & 31;
#pragma unroll 4
  for (int i = x.w0 + (threadIdx.x >> 5); i < x.w1; i += kWarps) {
    const uint32_t bits = pick(i);
    const int64_t to = place(i) + __popc(bits & ((1u << lane) - 1));
    if ((bits >> lane & 1) && to >= begin) out[to] = x.from + 32 * i + lane;
  }
}

// out[at .. end) = from, from + step, .. by so many CTAs, 16 bytes a store where they are aligned
__device__ __forceinline__ void fill(int32_t *out, int64_t at, int64_t end, int64_t from, int step, uint32_t rank, uint32_t ranks) {
  const int64_t threads = static_cast<int64_t>(ranks) * kThreads;
  if (at >= end) return;
  const int64_t head = min(end, at + static_cast<int64_t>((4 - (reinterpret_cast<uintptr_t>(out + at) >> 2 & 3)) & 3));
  const int64_t quads = (end - head) / 4;
  const auto value = [&](int64_t i) { return static_cast<int>(from + step * (i - at)); };
  const int64_t tid = static_cast<int64_t>(rank) * kThreads + threadIdx.x;
  for (int64_t q = tid; q < quads; q += threads) {
    const int64_t i = head + 4 * q;
    *reinterpret_cast<int4 *>(out + i) = make_int4(value(i), value(i + 1), value(i + 2), value(i + 3));
  }
  for (int64_t i = at + tid; i < head; i += threads) out[i] = value(i);
  for (int64_t i = head + 4 * quads + tid; i < end; i += threads) out[i] = value(i);
}

// The free list from such words, as far as it does not lie over them: every CTA counts the bits before its own words for itself.
__global__ void __launch_bounds__(kThreads, 1) list_free_kernel(ReleaseArgs p, const uint32_t *words, int count) {
  __shared__ int s_sum[3][kWarps];
  __shared__ uint2 s_word[kThreads];   // a word's open bits, and where its first goes
  sm100::grid_dependency_wait();
  sm100::grid_launch_dependents();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = ((count + static_cast<int>(gridDim.x) - 1) / static_cast<int>(gridDim.x) + 3) & ~3;   // at most kThreads (by the caller)
  const int w0 = min(count, static_cast<int>(blockIdx.x) * per), w1 = min(count, w0 + per);
  int before = 0, all = 0;
#pragma unroll 4
  for (int i = 4 * tid; i < count; i += 4 * kThreads) {   // (bits behind the last id are clear)
    const uint4 y = __ldcg(reinterpret_cast<const uint4 *>(words + i));
    const int n = __popc(y.x) + __popc(y.y) + __popc(y.z) + __popc(y.w);
    all += n;
    if (i < w0) before += n;
  }
  const int w = w0 + tid, left = p.num_pages - 32 * w;
  const uint32_t open = w >= w1 ? 0u : ~__ldcg(words + w) & (left >= 32 ? ~0u : left > 0 ? (1u << left) - 1 : 0u);
  const int n = __popc(open), inc = warp_scan(n, lane);
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    before += __shfl_xor_sync(0xffffffffu, before, o);
    all += __shfl_xor_sync(0xffffffffu, all, o);
  }
  if (lane == 31) {
    s_sum[0][warp] = before;
    s_sum[1][warp] = all;
    s_sum[2][warp] = inc;
  }
  __syncthreads();
  // (as many warps as lanes)
  const int of_warp = s_sum[2][lane], up_to = warp_scan(of_warp, lane);
  before = warp_scan(s_sum[0][lane], lane);
  all = warp_scan(s_sum[1][lane], lane);
  const int at = min(32 * w0, p.num_pages) - __shfl_sync(0xffffffffu, before, 31) + __shfl_sync(0xffffffffu, up_to - of_warp, warp) + inc - n;
  const int free = p.num_pages - __shfl_sync(0xffffffffu, all, 31);
  const int end = static_cast<int>(reinterpret_cast<const int32_t *>(words) - p.free_pages);
  s_word[tid] = make_uint2(open, at);
  __syncthreads();
#pragma unroll 4
  for (int i = warp; i < w1 - w0; i += kWarps) {   // a word's ids by a warp
    const uint2 x = s_word[i];
    const int to = static_cast<int>(x.y) + __popc(x.x & ((1u << lane) - 1));
    if ((x.x >> lane & 1) && to < end) p.free_pages[to] = 32 * (w0 + i) + lane;
  }
  fill(p.free_pages, free, end, -1, 0, blockIdx.x, gridDim.x);
  if (blockIdx.x == 0 && tid == 0) *p.num_free = free;
}

// `words`: the marks of all pages, where the whole GPU made them; the list lacks what lies over them
__global__ void __launch_bounds__(kThreads, 1) release_requests_kernel(ReleaseArgs p, int most, const uint32_t *words) {
  extern __shared__ uint32_t s_words[];
  __shared__ uint32_t s_warp[kWarps];
  const int tid = threadIdx.x;
  const uint32_t rank = cluster_rank();
  sm100::grid_dependency_wait();
  sm100::grid_launch_dependents();
  const int begin = words ? static_cast<int>(reinterpret_cast<const int32_t *>(words) - p.free_pages) : 0;
  if (words && __ldcg(p.num_free) <= begin) {
    fill(p.free_pages, begin, p.num_pages, -1, 0, rank, cluster_size());
    return;
  }
  if (!words) {
    for (int i = rank * kThreads + tid; i < p.num_rows; i += cluster_size() * kThreads)
      end_request(p.seq_lens, p.rows[i], p.t.B, p.t.status);
    cluster_sync();
  }
  int64_t done = 0;
  // (one window at least: the table is looked at where there are no pages, too)
  for (int64_t from = 0; from == 0 || from < p.num_pages; from += 32 * most) {
    const Window x = words ? marked(words, p.num_pages, most, s_words, s_warp, rank)
                           : mark(p.t, p.seq_lens, p.num_pages, static_cast<int>(from), most, s_words, s_warp, rank, from == 0);
    write_ids(
        x, p.free_pages,
        [&](int i) {
          const int left = x.span - 32 * i;
          return ~x.bits[i] & (left >= 32 ? ~0u : (1u << left) - 1);
        },
        [&](int i) { return done + 32 * i - x.before[i]; }, begin);
    done += x.span - x.set;
    cluster_sync();   // (the bits have been read)
  }
  fill(p.free_pages, max(done, static_cast<int64_t>(begin)), p.num_pages, -1, 0, rank, cluster_size());
  if (rank == 0 && tid == 0) *p.num_free = static_cast<int>(done);
}

__global__ void __launch_bounds__(kThreads, 1) compact_pages_kernel(CompactArgs p, int most, const uint32_t *words) {
  extern __shared__ uint32_t s_words[];
  __shared__ uint32_t s_warp[kWarps];
  const uint32_t rank = cluster_rank();
  sm100::grid_dependency_wait();
  sm100::grid_launch_dependents();
  const bool once = p.num_pages <= 32 * most;
  Window x{};
  int64_t set = 0;
  for (int64_t from = 0; from == 0 || from < p.num_pages; from += 32 * most) {
    x = words ? marked(words, p.num_pages, most, s_words, s_warp, rank)
              : mark(p.t, p.seq_lens, p.num_pages, static_cast<int>(from), most, s_words, s_warp, rank, from == 0);
    set += x.set;
    if (!once) cluster_sync();
  }
  const int used = static_cast<int>(set);   // pages in use: those of id `used` and above move
  // bits of a word whose first id is `id` that lie below it
  const auto below = [&](int id) { return used - id >= 32 ? ~0u : used <= id ? 0u : (1u << (used - id)) - 1; };
  int64_t ones = 0, stay = 0, holes = 0;    // set before the window; set below `used`, and clear, as far as the windows went
  for (int64_t from = 0; from == 0 || from < p.num_pages; from += 32 * most) {
    if (!once) x = mark(p.t, p.seq_lens, p.num_pages, static_cast<int>(from), most, s_words, s_warp, rank, false);
    const int in = min(max(used - x.from, 0), x.span);   // ids of the window below `used`
    const int64_t first_hole = holes, first_one = ones;
    if (in > 0) {
      const int w = in >> 5;
      const int kept = w < x.words ? static_cast<int>(x.before[w]) + __popc(x.bits[w] & ((1u << (in & 31)) - 1)) : x.set;
      stay += kept;
      holes += in - kept;
    }
    write_ids(
        x, p.copy_dst, [&](int i) { return ~x.bits[i] & below(x.from + 32 * i); },
        [&](int i) { return first_hole + 32 * i - x.before[i]; });
    write_ids(
        x, p.copy_src, [&](int i) { return x.bits[i] & ~below(x.from + 32 * i); },
        [&](int i) {   // (a word across `used` counts its own bits below it)
          return first_one + x.before[i] + __popc(x.bits[i] & below(x.from + 32 * i)) - stay;
        });
    ones += x.set;
    cluster_sync();   // the bits have been read, and the lists are there for all
  }
  const int copies = static_cast<int>(holes);
  pieces_of(p.t, p.seq_lens, rank, cluster_size(), false, [&](int row, int first, int n, const int (&id)[kPiece / 32]) {
    const int lane = threadIdx.x & 31;
    int32_t *to = p.new_table + row * p.new_stride + first;
    int y[kPiece / 32];
#pragma unroll
    for (int i = 0; i < kPiece / 32; ++i) {
      y[i] = id[i];
      if (32 * i + lane >= n || id[i] < used || id[i] >= p.num_pages) continue;
      int at = 0;   // its number among the ids that move
      if (once) {
        const int w = id[i] >> 5;
        at = static_cast<int>(x.before[w]) + __popc(x.bits[w] & ((1u << (id[i] & 31)) - 1)) - static_cast<int>(stay);
      } else {
        int hi = copies - 1;
        while (at < hi) {
          const int mid = (at + hi) >> 1;
          if (__ldcg(p.copy_src + mid) < id[i]) at = mid + 1; else hi = mid;
        }
      }
      if (at < copies) y[i] = __ldcg(p.copy_dst + at);
    }
#pragma unroll
    for (int i = 0; i < kPiece / 32; ++i)
      if (32 * i + lane < n) to[32 * i + lane] = y[i];
  });
  fill(p.copy_src, copies, p.room, -1, 0, rank, cluster_size());
  fill(p.copy_dst, copies, p.room, -1, 0, rank, cluster_size());
  const int64_t open = p.num_pages - set;
  fill(p.free_pages, 0, open, used, 1, rank, cluster_size());
  fill(p.free_pages, open, p.num_pages, -1, 0, rank, cluster_size());
  if (rank == 0 && threadIdx.x == 0) *p.num_free = static_cast<int>(open);
}

// Places of the table up to which one CTA, or four, have fewer meetings to pay for than loads.  Measured (release; tables of 2048,
// 8192, 32960 and 961536 places): one CTA 6.4, 9.5, 16.8 and 271 us, four 7.5, 8.3, 10.0 and 83, sixteen 8.9, 9.2, 10.0 and 35.
constexpr int64_t kPlacesOfOne = 1 << 12, kPlacesOfFour = 1 << 14;
// Places from which on all SMs mark (where a window holds all ids).  Release, then compact, with a cluster against with all SMs: 64000 places
// 9.5 and 10 (13.7 and 14.5) us, 131072 11.3 and 9.2 (17.1 and 16.3), 256000 16.7 and 11.2 (26 and 24), 512000 28 and 13 (45 and 37).
constexpr int64_t kPlacesOfAll = 1 << 17;

constexpr int kListCtas = 152;
static_assert((kMostWords + kListCtas - 1) / kListCtas + 3 <= kThreads, "a word of a CTA's a thread");
struct Ended {   // requests that end
  int32_t *seq_lens;
  const int32_t *rows;
  int num_rows;
};
template <typename K, typename A>
cudaError_t launch_marks(K kernel, std::mutex &mu, uint64_t &done, const A &a, const Ended &ended, cudaStream_t stream) {
  if (const cudaError_t e = set_attributes_once(mu, done, [&] {
        cudaError_t r = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 2 * 4 * kMostWords);
        if (r == cudaSuccess) r = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        return r;
      }))
    return e;
  const int words = static_cast<int>((static_cast<int64_t>(a.num_pages) + 31) / 32);
  const int most = words < kMostWords ? (words > 0 ? (words + 3) & ~3 : 4) : kMostWords;
  const int64_t places = static_cast<int64_t>(a.t.B) * a.t.width;
  const unsigned ranks = places <= kPlacesOfOne ? 1 : places <= kPlacesOfFour ? 4 : kMostRanks;
  uint32_t *marks = nullptr;
  if (places >= kPlacesOfAll && words <= most && a.num_pages >= most + 4) {
    // the last 16-byte words of the free list's memory, which is written behind their last use
    marks = reinterpret_cast<uint32_t *>(reinterpret_cast<uintptr_t>(a.free_pages + a.num_pages - most) & ~uintptr_t(15));
    const unsigned clears = static_cast<unsigned>(std::min<int64_t>(152, (std::max(most / 4, ended.num_rows) + 255) / 256));
    if (const cudaError_t e = launch_dependent(clear_marks_kernel, clears, 256, 0, stream, marks, most, ended.seq_lens, ended.rows,
                                               ended.num_rows, a.t.B, a.t.status))
      return e;
    if (const cudaError_t e = launch_dependent(mark_pages_kernel, 152, kThreads, 0, stream, a.t, static_cast<const int32_t *>(a.seq_lens),
                                               a.num_pages, marks))
      return e;
    if constexpr (std::is_same_v<A, ReleaseArgs>)
      if (const cudaError_t e = launch_dependent(list_free_kernel, kListCtas, kThreads, 0, stream, a, static_cast<const uint32_t *>(marks), words))
        return e;
  }
  return launch_dependent_clusters(kernel, ranks, ranks, kThreads, 2 * 4 * most, stream, a, most, static_cast<const uint32_t *>(marks));
}

// ---------------------------------------------------------------- copying
constexpr int kCopyThreads = 256, kCopyWarps = kCopyThreads / 32;
constexpr int kWindow = 4096;                       // pairs that a CTA lists at once
constexpr int kCopyPiece = 8192, kMostBuffers = 128;
struct CopyArgs {
  uint8_t *base[kMostBuffers];
  int64_t stride[kMostBuffers];
  int64_t bytes[kMostBuffers];
  int first[kMostBuffers + 1];   // pieces of the buffers before
  int buffers, same;             // same: pieces of every buffer, where they all have so many
  int num_pages, count;
  const int32_t *src, *dst;
  uint32_t *status;
};

__global__ void __launch_bounds__(kCopyThreads, 4) copy_pages_kernel(const __grid_constant__ CopyArgs p) {
  __shared__ int2 s_pair[kWindow];
  __shared__ int s_count[kCopyWarps];
  sm100::grid_dependency_wait();
  sm100::grid_launch_dependents();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int pieces = p.first[p.buffers];
  for (int c0 = 0; c0 < p.count; c0 += kWindow) {
    int pairs = 0;
    __syncthreads();
    for (int c = c0; c < min(p.count, c0 + kWindow); c += kCopyThreads) {
      const int i = c + tid;
      int2 x = make_int2(-1, -1);
      if (i < p.count) x = make_int2(p.src[i], p.dst[i]);
      bool on = x.x >= 0 && x.y >= 0;
      if (on && (x.x >= p.num_pages || x.y >= p.num_pages)) {
        if (blockIdx.x == 0) atomicOr(p.status, KDA_DEVICE_BAD_PAGE);
        on = false;
      }
      on = on && x.x != x.y;
      const uint32_t vote = __ballot_sync(0xffffffffu, on);
      if (lane == 0) s_count[warp] = __popc(vote);
      __syncthreads();
      int at = pairs + __popc(vote & ((1u << lane) - 1));
#pragma unroll
      for (int w = 0; w < kCopyWarps; ++w) {
        if (w < warp) at += s_count[w];
        pairs += s_count[w];
      }
      if (on) s_pair[at] = x;
      __syncthreads();
    }
    const int64_t units = static_cast<int64_t>(pairs) * pieces;
    for (int64_t u = blockIdx.x * kCopyWarps + warp; u < units; u += gridDim.x * kCopyWarps) {
      const int pair = static_cast<int>(u / pieces), r = static_cast<int>(u - static_cast<int64_t>(pair) * pieces);
      int buf;
      if (p.same) {
        buf = r / p.same;
      } else {
        int lo = 0, hi = p.buffers - 1;   // the last buffer with first <= r
        while (lo < hi) {
          const int mid = (lo + hi + 1) >> 1;
          if (p.first[mid] <= r) lo = mid; else hi = mid - 1;
        }
        buf = lo;
      }
      const int64_t off = static_cast<int64_t>(r - p.first[buf]) * kCopyPiece;
      const int n = static_cast<int>(min(static_cast<int64_t>(kCopyPiece), p.bytes[buf] - off)) / 16;
      const int2 x = s_pair[pair];
      const uint4 *from = reinterpret_cast<const uint4 *>(p.base[buf] + x.x * p.stride[buf] + off);
      uint4 *to = reinterpret_cast<uint4 *>(p.base[buf] + x.y * p.stride[buf] + off);
      if (n == kCopyPiece / 16) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint4 v[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) v[j] = __ldcs(from + h * 256 + j * 32 + lane);
#pragma unroll
          for (int j = 0; j < 8; ++j) __stcs(to + h * 256 + j * 32 + lane, v[j]);
        }
      } else {
        for (int e = lane; e < n; e += 32) to[e] = from[e];
      }
    }
  }
}

}  // namespace

cudaError_t launch_fork_requests(const ForkArgs &a, cudaStream_t stream) {
  const int most = 4 * 152;
  return launch_dependent(fork_requests_kernel, static_cast<unsigned>(a.forks < 1 ? 1 : a.forks < most ? a.forks : most), kForkThreads, 0,
                          stream, a);
}

cudaError_t launch_release_requests(const ReleaseArgs &a, cudaStream_t stream) {
  static std::mutex mu;
  static uint64_t done = 0;
  return launch_marks(release_requests_kernel, mu, done, a, Ended{a.seq_lens, a.rows, a.num_rows}, stream);
}

cudaError_t launch_compact_pages(const CompactArgs &a, cudaStream_t stream) {
  static std::mutex mu;
  static uint64_t done = 0;
  return launch_marks(compact_pages_kernel, mu, done, a, Ended{nullptr, nullptr, 0}, stream);
}

cudaError_t launch_copy_pages(const kda_page_buffer *buffers, int num_buffers, int num_pages, const int32_t *src,
                              const int32_t *dst, int count, uint32_t *status, cudaStream_t stream) {
  for (int b0 = 0; b0 < num_buffers; b0 += kMostBuffers) {
    CopyArgs a{};
    a.buffers = num_buffers - b0 < kMostBuffers ? num_buffers - b0 : kMostBuffers;
    int64_t pieces = 0;
    for (int i = 0; i < a.buffers; ++i) {
      const kda_page_buffer &b = buffers[b0 + i];
      a.base[i] = static_cast<uint8_t *>(b.base);
      a.stride[i] = b.page_stride;
      a.bytes[i] = b.bytes;
      a.first[i] = static_cast<int>(pieces);
      pieces += (b.bytes + kCopyPiece - 1) / kCopyPiece;
    }
    a.first[a.buffers] = static_cast<int>(pieces);
    a.same = a.first[1];
    for (int i = 1; i < a.buffers; ++i)
      if (a.first[i + 1] - a.first[i] != a.same) a.same = 0;
    a.num_pages = num_pages;
    a.count = count;
    a.src = src;
    a.dst = dst;
    a.status = status;
    const int64_t units = static_cast<int64_t>(count) * pieces, ctas = (units + kCopyWarps - 1) / kCopyWarps;
    if (units == 0) continue;
    const cudaError_t e = launch_dependent(copy_pages_kernel, static_cast<unsigned>(ctas < 4 * 152 ? ctas : 4 * 152), kCopyThreads, 0,
                                           stream, a);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace kda
