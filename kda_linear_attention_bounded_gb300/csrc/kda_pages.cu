// The pages' own operations: requests forked and ended, the cache compacted, pages copied.  Pages in use are those that the
// table's rows hold in their first ceil(length / page) places; nothing is counted from call to call.
//
// Forking.  Fork i needs a page where its parent's length n is no multiple of the page, and takes the free list's entry at the
// number of forks before it that need one.  Every CTA counts them for itself, in windows of a fork a thread, and then copies the
// rows of its own forks.  Bound by latency: lengths, counts, rows.
//
// Ending and compacting.  One cluster of CTAs has a bit for each page in each of its CTAs' shared memory (in windows of the ids
// where there are more).  Its warps take the rows in pieces of 512 places and set the bits of what they hold, each in its own
// CTA's bits (where a prompt's pages are held by many rows, most find their bit set).  Then each CTA joins an equal part of the
// words through the cluster, counts, and after the counts have gone round writes its part of the lists: places in a list are
// sums of bits, so the lists are in ascending order whatever came first.  With n pages in use, the i-th one of id n or above goes
// to the i-th free id below n.  A place of the table finds the number of its id in the list of ids that move, which is sorted.
//
// Copying.  Bound by HBM.  Every CTA lists the pairs of a window that are copies; pieces of 8 KB of them all stand in one line, of
// which each warp takes every so-manieth.
#include <climits>

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
  __shared__ int s_len[kForkThreads], s_parent[kForkThreads], s_child[kForkThreads], s_taken[kForkThreads];
  __shared__ int s_warp[kWarps];
  sm100::grid_dependency_wait();
  sm100::grid_launch_dependents();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int64_t before = 0;   // pages that the forks before the window need
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
    int64_t taken = before + __popc(on & ((1u << lane) - 1));
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) taken += s_warp[w];
      before += s_warp[w];
    }
    if (need && taken >= p.num_free) {
      bad |= KDA_DEVICE_NO_PAGES;
      child = -1;
    }
    if (bad && blockIdx.x == 0) atomicOr(p.t.status, bad);
    s_len[tid] = len;
    s_parent[tid] = parent;
    s_child[tid] = child;
    s_taken[tid] = need ? static_cast<int>(min(taken, static_cast<int64_t>(INT_MAX))) : -1;
    __syncthreads();
    for (int j = (blockIdx.x + gridDim.x - f0 % gridDim.x) % gridDim.x; j < kForkThreads && f0 + j < p.forks; j += gridDim.x) {
      const int c = s_child[j], n = s_len[j], at = s_taken[j];
      if (c < 0) {
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
          dst = p.free_pages[at];
          to[whole] = dst;
          if (src < 0 || dst < 0) atomicOr(p.t.status, KDA_DEVICE_BAD_PAGE);   // (no copy is made)
        }
        p.copy_src[f0 + j] = src;
        p.copy_dst[f0 + j] = dst;
        p.seq_lens[c] = n;
      }
    }
  }
  if (blockIdx.x == 0 && tid == 0) *p.pages_used = static_cast<int>(min(before, static_cast<int64_t>(p.num_free)));
}

// ---------------------------------------------------------------- pages in use
constexpr int kThreads = 1024, kWarps = kThreads / 32;
constexpr int kRanks = 8;                   // CTAs of the cluster
constexpr int kMostWords = 48 * 1024;       // words of bits (192 KB): windows of 1.5 M ids
constexpr int kPiece = 512;                 // places of a row that a warp takes

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
// A word of the shared memory of the cluster's CTA `rank`, at this CTA's address of it.
__device__ __forceinline__ uint32_t peer_word(const uint32_t *p, uint32_t rank) {
  uint32_t at, v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(sm100::smem_u32(p)), "r"(rank));
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
  return v;
}

// The table's pieces in turn: f(place of the table's row, its row, places) of each by a warp of the cluster.
template <typename F>
__device__ __forceinline__ void pieces_of(const TableArgs &t, const int32_t *seq_lens, uint32_t rank, bool record, F f) {
  const int lane = threadIdx.x & 31, w = rank * kWarps + (threadIdx.x >> 5);
  const int per_row = max(1, (t.width + kPiece - 1) / kPiece);
  const int64_t units = static_cast<int64_t>(per_row) * t.B;
  for (int64_t u = w; u < units; u += kRanks * kWarps) {
    const int piece = static_cast<int>(u / t.B), b = static_cast<int>(u - static_cast<int64_t>(piece) * t.B);
    const int pages = pages_of(t, __ldcg(seq_lens + b), record && piece == 0 && lane == 0);
    const int first = piece * kPiece, n = min(kPiece, pages - first);
    if (n > 0) f(b, first, n, lane);
  }
}

// Sets the bits of the window's ids that the rows hold, joined over the cluster: afterwards words w0 .. w1 of `bits` hold the
// whole cluster's.  Bits behind the window's last id are set, so that they are no free pages.
__device__ __forceinline__ void mark(const TableArgs &t, const int32_t *seq_lens, int num_pages, int window, int words, uint32_t *bits,
                                     uint32_t rank, bool record, int w0, int w1) {
  const int tid = threadIdx.x;
  for (int i = tid; i < words; i += kThreads) bits[i] = 0;
  __syncthreads();
  const uint32_t span = min(words * 32, num_pages - window);
  pieces_of(t, seq_lens, rank, record, [&](int b, int first, int n, int lane) {
    const int32_t *row = t.table + b * t.stride + first;
#pragma unroll 1
    for (int e0 = 0; e0 < n; e0 += 128) {
      int id[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int e = e0 + 32 * j + lane;
        id[j] = e < n ? row[e] : -2;
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (id[j] == -2 && e0 + 32 * j + lane >= n) continue;
        if (id[j] < 0 || id[j] >= num_pages) {
          if (record) atomicOr(t.status, KDA_DEVICE_BAD_PAGE);
          continue;
        }
        const uint32_t at = static_cast<uint32_t>(id[j] - window);
        if (id[j] < window || at >= span) continue;
        const uint32_t bit = 1u << (at & 31);
        volatile uint32_t *word = bits + (at >> 5);
        if (!(*word & bit)) atomicOr(bits + (at >> 5), bit);
      }
    }
  });
  cluster_sync();
  for (int i = w0 + tid; i < w1; i += kThreads) {
    uint32_t x[kRanks];
#pragma unroll
    for (uint32_t r = 0; r < kRanks; ++r) x[r] = peer_word(bits + i, r);
#pragma unroll
    for (uint32_t r = 1; r < kRanks; ++r) x[0] |= x[r];
    const int valid = static_cast<int>(span) - 32 * i;
    if (valid < 32) x[0] |= valid <= 0 ? ~0u : ~0u << valid;
    bits[i] = x[0];   // (no other CTA reads these words of this CTA's)
  }
  __syncthreads();
}

// Ids of the window that `pick(word, its first id)` has bits for, among this CTA's words: counted, or (Emit) written in order
// from out[base] on.
template <bool kEmit, typename P>
__device__ __forceinline__ int pick_ids(const uint32_t *bits, int w0, int w1, int window, int *s_warp, int32_t *out, int64_t base, P pick) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int total = 0;
  for (int i0 = w0; i0 < w1; i0 += kThreads) {
    const int i = i0 + tid;
    const uint32_t x = i < w1 ? pick(bits[i], window + 32 * i) : 0;
    const int n = __popc(x), inc = warp_scan(n, lane);
    if (lane == 31) s_warp[warp] = inc;
    __syncthreads();
    int mine = 0, all = 0;
#pragma unroll 8
    for (int w = 0; w < kWarps; ++w) {
      const int c = s_warp[w];
      mine += w < warp ? c : 0;
      all += c;
    }
    if (kEmit && __any_sync(0xffffffffu, n)) {
      const int at = mine + inc - n;
#pragma unroll 1
      for (int j = 0; j < 32; ++j) {
        const uint32_t y = __shfl_sync(0xffffffffu, x, j);
        const int before = __shfl_sync(0xffffffffu, at, j);
        if (y >> lane & 1)
          out[base + total + before + __popc(y & ((1u << lane) - 1))] = window + 32 * (i0 + 32 * warp + j) + lane;
      }
    }
    total += all;
    __syncthreads();
  }
  return total;
}

// Sums of every CTA's counts before this one's, and of all.  (Counts are written by one thread; the caller synchronises before
// they are written again.)
__device__ __forceinline__ void exchange(uint32_t *s_count, int count, uint32_t rank, int64_t &before, int64_t &all) {
  if (threadIdx.x == 0) *s_count = count;
  cluster_sync();
  before = all = 0;
#pragma unroll
  for (uint32_t r = 0; r < kRanks; ++r) {
    const uint32_t c = peer_word(s_count, r);
    before += r < rank ? c : 0;
    all += c;
  }
}

struct Part {   // of the bits: this CTA's words of a window
  int words, w0, w1;
};
__device__ __forceinline__ Part part_of(int num_pages, int window, int most, uint32_t rank) {
  Part x;
  x.words = min(most, (num_pages - window + 31) / 32);
  const int per = (x.words + kRanks - 1) / kRanks;
  x.w0 = min(x.words, static_cast<int>(rank) * per);
  x.w1 = min(x.words, x.w0 + per);
  return x;
}

__global__ void __launch_bounds__(kThreads, 1) release_requests_kernel(ReleaseArgs p, int most_words) {
  extern __shared__ uint32_t s_bits[];
  __shared__ int s_warp[kWarps];
  __shared__ uint32_t s_count;
  const int tid = threadIdx.x;
  const uint32_t rank = cluster_rank();
  sm100::grid_dependency_wait();
  sm100::grid_launch_dependents();
  for (int i = rank * kThreads + tid; i < p.num_rows; i += kRanks * kThreads) {
    const int row = p.rows[i];
    if (row >= p.t.B) atomicOr(p.t.status, KDA_DEVICE_BAD_INDEX);
    else if (row >= 0) p.seq_lens[row] = 0;
  }
  cluster_sync();
  int64_t done = 0;
  for (int64_t from = 0; from < p.num_pages; from += 32 * most_words) {
    const int window = static_cast<int>(from);
    const Part x = part_of(p.num_pages, window, most_words, rank);
    mark(p.t, p.seq_lens, p.num_pages, window, x.words, s_bits, rank, window == 0, x.w0, x.w1);
    const auto open = [](uint32_t word, int) { return ~word; };
    const int mine = pick_ids<false>(s_bits, x.w0, x.w1, window, s_warp, nullptr, 0, open);
    int64_t before, all;
    exchange(&s_count, mine, rank, before, all);
    pick_ids<true>(s_bits, x.w0, x.w1, window, s_warp, p.free_pages, done + before, open);
    done += all;
    cluster_sync();   // (counts and bits have been read)
  }
  for (int64_t i = done + rank * kThreads + tid; i < p.num_pages; i += kRanks * kThreads) p.free_pages[i] = -1;
  if (rank == 0 && tid == 0) *p.num_free = static_cast<int>(done);
}

__global__ void __launch_bounds__(kThreads, 1) compact_pages_kernel(CompactArgs p, int most_words) {
  extern __shared__ uint32_t s_bits[];
  __shared__ int s_warp[kWarps];
  __shared__ uint32_t s_count[3];
  const int tid = threadIdx.x;
  const uint32_t rank = cluster_rank();
  sm100::grid_dependency_wait();
  sm100::grid_launch_dependents();
  const bool once = p.num_pages <= 32 * most_words;
  // pages in use
  int64_t open = 0;
  for (int64_t from = 0; from < p.num_pages; from += 32 * most_words) {
    const int window = static_cast<int>(from);
    const Part x = part_of(p.num_pages, window, most_words, rank);
    mark(p.t, p.seq_lens, p.num_pages, window, x.words, s_bits, rank, window == 0, x.w0, x.w1);
    const int mine = pick_ids<false>(s_bits, x.w0, x.w1, window, s_warp, nullptr, 0, [](uint32_t word, int) { return ~word; });
    int64_t before, all;
    exchange(s_count, mine, rank, before, all);
    open += all;
    if (!once) cluster_sync();
  }
  const int used = static_cast<int>(p.num_pages - open);
  // bits of a word whose first id is `id` that lie below the number of pages in use
  const auto below = [&](int id) { return used - id >= 32 ? ~0u : used <= id ? 0u : (1u << (used - id)) - 1; };
  const auto hole = [&](uint32_t word, int id) { return ~word & below(id); };
  const auto moves = [&](uint32_t word, int id) {
    const int left = p.num_pages - id;   // (bits behind the last id are set)
    return word & ~below(id) & (left >= 32 ? ~0u : (1u << left) - 1);
  };
  int64_t holes = 0, moved = 0;
  for (int64_t from = 0; from < p.num_pages; from += 32 * most_words) {
    const int window = static_cast<int>(from);
    const Part x = part_of(p.num_pages, window, most_words, rank);
    if (!once) mark(p.t, p.seq_lens, p.num_pages, window, x.words, s_bits, rank, false, x.w0, x.w1);
    const int h = pick_ids<false>(s_bits, x.w0, x.w1, window, s_warp, nullptr, 0, hole);
    const int m = pick_ids<false>(s_bits, x.w0, x.w1, window, s_warp, nullptr, 0, moves);
    int64_t h0, h1, m0, m1;
    exchange(s_count + 1, h, rank, h0, h1);
    exchange(s_count + 2, m, rank, m0, m1);
    pick_ids<true>(s_bits, x.w0, x.w1, window, s_warp, p.copy_dst, holes + h0, hole);
    pick_ids<true>(s_bits, x.w0, x.w1, window, s_warp, p.copy_src, moved + m0, moves);
    holes += h1;
    moved += m1;
    cluster_sync();   // counts and bits have been read, and the lists are there for all
  }
  const int copies = static_cast<int>(moved);
  const int at = rank * kThreads + tid, step = kRanks * kThreads;
  pieces_of(p.t, p.seq_lens, rank, false, [&](int b, int first, int n, int lane) {
    const int32_t *row = p.t.table + b * p.t.stride + first;
    int32_t *to = p.new_table + b * p.new_stride + first;
#pragma unroll 4
    for (int e = lane; e < n; e += 32) {
      int id = row[e];
      if (id >= used && id < p.num_pages) {
        int lo = 0, hi = copies - 1;   // its number among the ids that move
        while (lo < hi) {
          const int mid = (lo + hi) >> 1;
          if (__ldcg(p.copy_src + mid) < id) lo = mid + 1; else hi = mid;
        }
        if (lo < copies) id = __ldcg(p.copy_dst + lo);
      }
      to[e] = id;
    }
  });
  for (int i = copies + at; i < p.room; i += step) p.copy_src[i] = p.copy_dst[i] = -1;
  for (int i = at; i < p.num_pages; i += step) p.free_pages[i] = i < open ? used + i : -1;
  if (at == 0) *p.num_free = static_cast<int>(open);
}

template <typename K, typename A>
cudaError_t launch_marks(K kernel, std::mutex &mu, uint64_t &done, const A &a, cudaStream_t stream) {
  if (const cudaError_t e = set_attributes_once(mu, done, [&] {
        return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 4 * kMostWords);
      }))
    return e;
  const int words = static_cast<int>((static_cast<int64_t>(a.num_pages) + 31) / 32);
  const int most = words < kMostWords ? (words > 0 ? words : 1) : kMostWords;
  return launch_dependent_clusters(kernel, kRanks, kRanks, kThreads, 4 * most, stream, a, most);
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
  return launch_marks(release_requests_kernel, mu, done, a, stream);
}

cudaError_t launch_compact_pages(const CompactArgs &a, cudaStream_t stream) {
  static std::mutex mu;
  static uint64_t done = 0;
  return launch_marks(compact_pages_kernel, mu, done, a, stream);
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
