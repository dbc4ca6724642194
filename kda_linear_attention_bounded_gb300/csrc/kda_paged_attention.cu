// Attention of new tokens over a paged key-value cache, split over the cache's length and joined.
//
// Request b has len_b tokens in its pages, the last T of them new.  Row (t, g) of key head h is query head
// h (Hq / Hk) + g of new token t and sees the tokens j < n_t = len_b - T + t + 1:
//   s_j = scale q . k_j,   m = max s_j,   l = sum e^(s_j - m),   o = sum e^(s_j - m) v_j / l,   lse = m + log l
// One pass over the tokens with running m, l and o (fp32); parts over disjoint tokens join as
//   m = max m_p,  l = sum e^(m_p - m) l_p,  o = sum e^(m_p - m) l_p o_p / l.
//
// Bound by HBM: each token costs 512 bytes per key head and only 4 Hq / Hk T 128 operations.  So the work is cut by
// bytes: the tiles of 64 tokens of every (request, key head, row block) stand in one line, of which each CTA (two per
// SM, a fixed grid) takes an equal stretch, whatever the lengths are.  In the line an item takes kItemCost units, for its
// queries and its end, and one for each tile; a tile is the stretch's that its unit is in.  (Measured: 64 requests of 1
// to 8192 tokens 61 us without, 55 us with 2 to 6, where stretches of many short requests had come last.)  A stretch that begins or ends inside an item
// leaves its part (m, l, o) in the workspace; a second kernel, launched as a programmatic dependent, joins an item's
// parts in the order of its tokens, so results do not depend on timing.  Few short items go to a cluster of CTAs each
// instead, which join in shared memory.
//
// One warp, or two, bring tiles through three 32 KB stages (page ids are looked up a tile earlier), four compute on them,
// and they meet at mbarriers only.  Pages whose size has a power of two of 16 or more in it come by TMA, in boxes of so many
// rows (up to 64); other sizes by 16-byte asynchronous copies, by two warps.  A CTA's rows (16, 32 or 64 of
// them: query heads of the key head x new tokens) share every key and value; with 16 rows the four warps split a tile's
// tokens, with 64 its rows.  Products are mma.sync m16n8k16 (bf16, fp32 sums): even 64 rows need 64 operations per
// byte, which it sustains at HBM speed.  e^(s - m) is rounded to bf16 for the second product (the cache's own
// precision), l sums the unrounded.
#include <cuda.h>

#include <algorithm>

#include "kda_hybrid.cuh"

namespace kda {
namespace {

constexpr int kThreads = 192, kComputeWarps = 4;   // and two loading warps (the second for copies only)
constexpr int kTile = 64;        // tokens per tile
constexpr int kStages = 3;
constexpr uint32_t kStageBytes = 2 * kTile * kD * 2;   // K rows, then V rows
constexpr uint32_t kHalf = kTile * 128;                // 64 channels of a tile's rows (128-byte swizzle); K: 2, V: 2
constexpr uint32_t OFF_INFO = kStages * kStageBytes;   // int4 per stage: request, head and row block, tile, length
constexpr uint32_t OFF_MASK = OFF_INFO + 64;           // uint64 per stage: which tokens of the tile are there
constexpr uint32_t OFF_ML = OFF_MASK + 32;             // float [4 warps][16 rows][2]
constexpr uint32_t OFF_CML = OFF_ML + 512;             // float2 [64]: a cluster CTA's rows' maximum and sum of weights
constexpr uint32_t OFF_SCAN = OFF_CML + 512;
constexpr uint32_t OFF_BAR = OFF_SCAN + 64;            // landed [3], free [3], readers met, abort flag
constexpr uint32_t kSmemBytes = OFF_BAR + 64 + 1024;
static_assert(4 * 16 * kD * 4 <= kStageBytes, "the warps' sums fit one stage");
static_assert(16 * kStages <= 64 && 8 * kStages <= 32 && (2 * kStages + 1) * 8 <= 56, "small parts of the shared memory map");

// 16 bytes (8 channels) `chunk` of a tile's row
__device__ __forceinline__ uint32_t row_chunk(int row, int chunk) {
  return (chunk >> 3) * kHalf + row * 128 + (((chunk ^ row) & 7) << 4);
}

struct PagedMaps {
  CUtensorMap k, v;   // [page, token, head, 128], boxes of 64 channels x `box` tokens, 128-byte swizzle
  int box;            // 0: none, rows come by asynchronous copies
};

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap *map, int c0, int c1, int c2, int c3,
                                            uint64_t *bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];"
      ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(sm100::smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ void cp16(uint32_t dst, const void *src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// A shared-memory address of this CTA, in the cluster's CTA `rank`
__device__ __forceinline__ uint32_t peer(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ float2 peer_f2(uint32_t addr) {
  float2 v;
  asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ float4 peer_f4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr) : "memory");
  return v;
}
// The two of a word's bf16 that bits 0 and 1 ask for.
__device__ __forceinline__ uint32_t pick2(uint32_t bits) {
  return (bits & 1 ? 0x0000FFFFu : 0u) | (bits & 2 ? 0xFFFF0000u : 0u);
}
// Tokens 0 .. n - 1 of a tile.
__device__ __forceinline__ uint64_t first_tokens(int n) {
  return n <= 0 ? 0ull : n >= 64 ? ~0ull : (1ull << n) - 1;
}
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
// D (16x8 fp32) += A (16x16 bf16, row) * B (16x8 bf16, col)
__device__ __forceinline__ void mma_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// A place in the line of tiles: tile `tile` of item (request b, key head and row block hr).
struct Cursor {
  int b, hr, tile, ntiles, len;
  int next;       // length of the next request (looked up early)
  int cost;       // units of an item besides its tiles'
  int64_t unit;   // of the tile
};
constexpr uint32_t kMostRanks = 8;   // CTAs of a cluster
constexpr int kItemCost = 4;   // (0 where there is a CTA for every tile)
constexpr int kLastTile = 1 << 30;   // with the head and row block: the stretch ends here

// Tokens of request b; a length that is none, or that its table row cannot hold, counts as 0 (and is recorded, by the
// thread whose part it is).
__device__ __forceinline__ int request_len(const PagedArgs &p, int b, bool record = false) {
  const int len = p.seq_lens[b];
  if (len < 0 || len > p.max_len) {
    if (record) atomicOr(p.status, KDA_DEVICE_BAD_COUNT);
    return 0;
  }
  return len;
}
// Tiles of an item: an empty request keeps one (its rows are written as empty)
__device__ __forceinline__ int tile_count(int len) { return max(1, (len + kTile - 1) / kTile); }

__device__ __forceinline__ void advance(const PagedArgs &p, Cursor &c, int items_per_request) {
  ++c.unit;
  if (++c.tile < c.ntiles) return;
  c.tile = 0;
  c.unit += c.cost;
  if (++c.hr < items_per_request) return;
  c.hr = 0;
  ++c.b;
  c.len = c.next;
  c.ntiles = tile_count(c.len);
  if (c.b + 1 < p.B) c.next = request_len(p, c.b + 1);
}

// One output row (a new token's query head) by a warp, four channels a lane, from its sums.
__device__ __forceinline__ void paged_store_row(const PagedArgs &p, int b, int t, int head, int lane, float4 acc, float m,
                                                float l) {
  const int64_t row = static_cast<int64_t>(b) * p.T + t;
  const float inv = l == 0.f ? 0.f : 1.0f / l;   // a row that sees nothing: zeros
  *reinterpret_cast<uint2 *>(p.out + row * p.out_stride + static_cast<int64_t>(head) * kD + lane * 4) =
      make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
  if (p.lse && lane == 0) p.lse[row * p.Hk * p.G + head] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
}

// WR: row groups of 16; the other 4 / WR warps of a row group split the tile's tokens.  kCluster: a cluster an item (no
// joins), else stretches of the line.
template <int WR, bool kCluster>
__global__ void __launch_bounds__(kThreads, 2) paged_attention_kernel(PagedArgs p, const __grid_constant__ PagedMaps maps) {
  constexpr int WT = 4 / WR, kTok = kTile / WT, kNT = kTok / 8;
  constexpr int kRows = 16 * WR;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *sm = smem_raw + (-sm100::smem_u32(smem_raw) & 1023u);
  int4 *s_info = reinterpret_cast<int4 *>(sm + OFF_INFO);
  uint64_t *s_mask = reinterpret_cast<uint64_t *>(sm + OFF_MASK);
  float *s_ml = reinterpret_cast<float *>(sm + OFF_ML);
  uint64_t *landed = reinterpret_cast<uint64_t *>(sm + OFF_BAR), *freed = landed + kStages, *met = freed + kStages;
  volatile uint32_t *s_abort = reinterpret_cast<volatile uint32_t *>(sm + OFF_BAR + 56);
  const uint32_t smem = sm100::smem_u32(sm);
  const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  const int wr = warp % WR, wt = warp / WR;
  const int ipr = p.Hk * p.row_blocks;   // items per request
  if (maps.box && tid == 32 * kComputeWarps) {
    sm100::prefetch_tensormap(&maps.k);
    sm100::prefetch_tensormap(&maps.v);
  }
  if (tid == 0) {
    for (int i = 0; i < kStages; ++i) {
      sm100::mbar_init(&landed[i], maps.box ? 1 : 66);
      sm100::mbar_init(&freed[i], kComputeWarps);
    }
    sm100::mbar_init(met, kComputeWarps);
    *s_abort = 0;
    sm100::fence_mbar_init();
  }
  sm100::grid_dependency_wait();
  sm100::grid_launch_dependents();

  // ---- this CTA's stretch of the line of tiles
  int64_t *s_scan = reinterpret_cast<int64_t *>(sm + OFF_SCAN);   // [6] warp sums, then the start's request and tile
  int64_t first = 0, last = 0, total = 0;
  int stretches = 0;   // CTAs with units: every one of them has at least one
  Cursor cur;
  const uint32_t ranks = kCluster ? p.cluster : 1, rank = blockIdx.x % ranks;
  if constexpr (kCluster) {
    const int item = blockIdx.x / ranks;
    cur.b = item / ipr;
    cur.hr = item % ipr;
    cur.len = request_len(p, cur.b, tid == 0);
    cur.ntiles = tile_count(cur.len);
    cur.cost = 0;
    first = static_cast<int64_t>(cur.ntiles) * rank / ranks;
    last = static_cast<int64_t>(cur.ntiles) * (rank + 1) / ranks;
    cur.unit = first;
    cur.tile = static_cast<int>(first);
    __syncthreads();
  } else {
    const int per = (p.B + kThreads - 1) / kThreads;
    const int b0 = min(p.B, tid * per), b1 = min(p.B, b0 + per);
    int64_t sum = 0;
    for (int b = b0; b < b1; ++b) sum += tile_count(request_len(p, b, true));
    int64_t inc = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t u = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += u;
    }
    if (lane == 31) s_scan[warp] = inc;
    __syncthreads();
    int64_t before = inc - sum;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
      if (w < warp) before += s_scan[w];
      total += s_scan[w];
    }
    cur.cost = total * ipr > gridDim.x ? kItemCost : 0;
    total = (total + static_cast<int64_t>(cur.cost) * p.B) * ipr;
    before = (before + static_cast<int64_t>(cur.cost) * b0) * ipr;
    sum = (sum + static_cast<int64_t>(cur.cost) * (b1 - b0)) * ipr;
    stretches = static_cast<int>(min(total, static_cast<int64_t>(gridDim.x)));
    if (blockIdx.x < stretches) {
      first = total * blockIdx.x / stretches;
      last = total * (blockIdx.x + 1) / stretches;
    }
    // the thread whose requests hold the first tile walks to it
    if (first < last && first >= before && first < before + sum) {
      int b = b0;
      int64_t at = before;
      while (true) {
        const int64_t n = static_cast<int64_t>(cur.cost + tile_count(request_len(p, b))) * ipr;
        if (first < at + n) break;
        at += n;
        ++b;
      }
      s_scan[6] = b;
      s_scan[7] = first - at;
    }
    __syncthreads();
  }
  bool none = first >= last;
  if (!kCluster && !none) {
    cur.b = static_cast<int>(s_scan[6]);
    cur.len = request_len(p, cur.b);
    cur.ntiles = tile_count(cur.len);
    const int per_item = cur.cost + cur.ntiles;
    cur.hr = static_cast<int>(s_scan[7] / per_item);
    const int u = static_cast<int>(s_scan[7] - static_cast<int64_t>(cur.hr) * per_item);
    cur.tile = max(0, u - cur.cost);
    cur.unit = first - u + cur.cost + cur.tile;
    none = cur.unit >= last;   // (a stretch of an item's first units alone)
  }
  // an item that an earlier CTA began: the CTA at the first cut inside it describes the join
  if (!kCluster && tid == 0) {
    int4 j = make_int4(0, 0, 0, 0);
    if (!none && cur.tile > 0) {
      const int64_t begin = cur.unit - cur.tile, end = begin + cur.ntiles;   // the units of the item's tiles
      if (total * (blockIdx.x - 1) / stretches <= begin) {
        int n = 1;   // stretches behind the first that begin before the item's end
        while (blockIdx.x + n < stretches && total * (blockIdx.x + n) / stretches < end) ++n;
        j = make_int4(n + 1, cur.b, cur.hr, 0);
      }
    }
    p.joins[blockIdx.x] = j;
  }
  // A cluster's end: its CTAs' rows (channels in stage 0, maximum and weights beside) are joined in the order of their
  // tokens, each CTA taking every ranks-th row.  All threads of the cluster come here.
  const uint32_t c_rows = smem, c_ml = smem + OFF_CML;
  const auto finish = [&] {
    if (!kCluster || ranks == 1) return;
    if (none && tid < kRows) *reinterpret_cast<float2 *>(sm + OFF_CML + 8 * tid) = make_float2(-INFINITY, 0.f);
    cluster_sync();
    if (warp < kComputeWarps) {
      const int rb = cur.hr % p.row_blocks, h = cur.hr / p.row_blocks;
      for (int r = rank + ranks * warp; r < kRows; r += ranks * kComputeWarps) {
        const int row = rb * kRows + r, t = row / p.G;
        if (t >= p.T) break;
        float2 ml[kMostRanks];
        float4 x[kMostRanks];
        float mm = -INFINITY, ll = 0.f;
#pragma unroll
        for (uint32_t q = 0; q < kMostRanks; ++q) {
          ml[q] = make_float2(-INFINITY, 0.f);
          if (q < ranks) {
            ml[q] = peer_f2(peer(c_ml + 8 * r, q));
            x[q] = peer_f4(peer(c_rows + (r * kD + lane * 4) * 4, q));
          }
          mm = fmaxf(mm, ml[q].x);
        }
        const float bs = mm == -INFINITY ? 0.f : mm;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (uint32_t q = 0; q < kMostRanks; ++q)
          if (ml[q].x != -INFINITY || ml[q].y != 0.f) {   // (a CTA without tokens has written no channels)
            const float c = fast_exp2(ml[q].x - bs);
            ll += c * ml[q].y;
            acc.x += c * x[q].x; acc.y += c * x[q].y; acc.z += c * x[q].z; acc.w += c * x[q].w;
          }
        paged_store_row(p, cur.b, t, h * p.G + row % p.G, lane, acc, mm, ll);
      }
    }
    cluster_sync();   // (a CTA's shared memory stays while others read it)
  };
  if (none) {
    finish();
    return;
  }

  if (warp >= kComputeWarps) {
    // ---------------------------------------------------------------- loads
    const int box = maps.box ? maps.box : 1, boxes = kTile / box;
    const int half = warp - kComputeWarps;   // copies: rows 32 half + lane; TMA: the first warp's lanes have a box each
    if (half && maps.box) {
      finish();
      return;
    }
    cur.next = cur.b + 1 < p.B ? request_len(p, cur.b + 1) : 0;
    const int at = lane + 32 * half;
    int id = 0;
    bool there = false;
    auto ask = [&] {   // the pages of the tile at the cursor
      const int pos = cur.tile * kTile + at * box;
      there = at < boxes && pos < cur.len;
      id = there ? p.table[static_cast<int64_t>(cur.b) * p.table_stride + pos / p.page] : 0;
    };
    ask();
    for (int i = 0; ; ++i) {
      const int st = i % kStages, pos0 = cur.tile * kTile, h = cur.hr / p.row_blocks;
      const uint32_t dst = smem + st * kStageBytes;
      int4 info = make_int4(cur.b, cur.hr, cur.tile, cur.len);
      const int pg = id;
      const bool ok = there && pg >= 0 && pg < p.num_pages;
      if (there && !ok) atomicOr(p.status, KDA_DEVICE_BAD_PAGE);
      advance(p, cur, ipr);
      const bool more = cur.unit < last;
      if (more)
        ask();
      else
        info.y |= kLastTile;
      const uint32_t on = __ballot_sync(0xffffffffu, ok);
      if (i >= kStages) sm100::wait_or_abort(&freed[st], (i / kStages - 1) & 1, s_abort, p.status);
      if (__any_sync(0xffffffffu, *s_abort != 0)) break;   // (what was asked for lands below)
      if (lane == 0) {
        if (half == 0) s_info[st] = info;
        if (maps.box) {
          uint64_t mask = 0;
          for (int x = 0; x < boxes; ++x)
            if (on >> x & 1) mask |= first_tokens(box) << (x * box);
          s_mask[st] = mask & first_tokens(info.w - pos0);
          sm100::mbar_arrive_expect_tx(&landed[st], __popc(on) * box * 512);
        } else {
          reinterpret_cast<uint32_t *>(&s_mask[st])[half] = on;
          sm100::mbar_arrive(&landed[st]);
        }
      }
      __syncwarp();
      if (maps.box) {
        if (ok) {
          const int tok = (pos0 + lane * box) % p.page;
          const uint32_t to = dst + lane * box * 128;
          tma_load_4d(to, &maps.k, 0, h, tok, pg, &landed[st]);
          tma_load_4d(to + kHalf, &maps.k, 64, h, tok, pg, &landed[st]);
          tma_load_4d(to + 2 * kHalf, &maps.v, 0, h, tok, pg, &landed[st]);
          tma_load_4d(to + 3 * kHalf, &maps.v, 64, h, tok, pg, &landed[st]);
        }
        __syncwarp();
      } else {
        const int64_t tok = (pos0 + at) % p.page;   // this lane's row (-1: not there)
        const int64_t ka = ok ? pg * p.k_page_stride + tok * p.k_token_stride + h * p.k_head_stride : -1;
        const int64_t va = pg * p.v_page_stride + tok * p.v_token_stride + h * p.v_head_stride;
        const int chunk = lane & 15;
#pragma unroll 4
        for (int r = 0; r < 32; r += 2) {
          const int from = r + (lane >> 4);
          const int64_t k = __shfl_sync(0xffffffffu, ka, from), v = __shfl_sync(0xffffffffu, va, from);
          if (k >= 0) {
            const uint32_t to = dst + row_chunk(32 * half + from, chunk);
            cp16(to, p.k + k + chunk * 8);
            cp16(to + 2 * kHalf, p.v + v + chunk * 8);
          }
        }
        asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(sm100::smem_u32(&landed[st])) : "memory");
      }
      if (!more) break;
    }
    // (after a timeout the copies in flight are waited for here; otherwise the readers have waited for them)
    asm volatile("cp.async.wait_all;" ::: "memory");
    if (*s_abort)
      for (int i = 0; i < kStages; ++i) {
        sm100::mbar_wait(&landed[i], 0);
        sm100::mbar_wait(&landed[i], 1);
      }
    __syncwarp();
    finish();
    return;
  }

  // ------------------------------------------------------------------ products
  const float sl2 = p.scale * kLog2e;
  uint32_t qf[8][4];
  float o[16][4], m2[2], l2[2];   // rows g and g + 8 of the warp's group
  int lim[2];                     // tokens each row sees
  const int g = lane >> 2, t4 = lane & 3;
  bool fresh = true;              // an item begins
  int begun = 0;                  // the stretch's first tile of the item
  uint32_t meetings = 0;
  // the readers wait for each other (bounded like every wait: after a timeout nobody is waited for)
  const auto meet = [&] {
    __syncwarp();
    if (lane == 0) sm100::mbar_arrive(met);
    sm100::wait_or_abort(met, meetings++ & 1, s_abort, p.status);
  };

  const auto begin_item = [&] {
    const int rb = cur.hr % p.row_blocks, h = cur.hr / p.row_blocks;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const int row = rb * kRows + 16 * wr + g + 8 * s;   // row of the key head: new token row / G, head row % G
      const int t = row / p.G;
      lim[s] = t < p.T ? min(max(cur.len - p.T + t + 1, 0), cur.len) : 0;
      const uint16_t *src = p.q + (static_cast<int64_t>(cur.b) * p.T + t) * p.q_stride + (h * p.G + row % p.G) * kD + t4 * 2;
#pragma unroll
      for (int kk = 0; kk < 8; ++kk) {
        qf[kk][s] = t < p.T ? *reinterpret_cast<const uint32_t *>(src + kk * 16) : 0u;
        qf[kk][s + 2] = t < p.T ? *reinterpret_cast<const uint32_t *>(src + kk * 16 + 8) : 0u;
      }
      m2[s] = -INFINITY;
      l2[s] = 0.f;
    }
#pragma unroll
    for (int n = 0; n < 16; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[n][e] = 0.f;
  };
  begin_item();   // (the first one's queries come beside its first tile)
  for (int i = 0;; ++i) {
    const int st = i % kStages;
    sm100::wait_or_abort(&landed[st], (i / kStages) & 1, s_abort, p.status);
    const int4 info = s_info[st];
    if (__any_sync(0xffffffffu, *s_abort != 0)) break;
    cur.b = info.x; cur.hr = info.y & (kLastTile - 1); cur.tile = info.z; cur.len = info.w;
    const bool stretch_ends = info.y & kLastTile;
    if (fresh) {
      fresh = false;
      begun = i;
      if (i > 0) begin_item();
    }
    const uint32_t kt = smem + st * kStageBytes, vt = kt + 2 * kHalf;
    const int tok0 = wt * kTok;   // the warp's tokens of the tile

    // ---- scores
    float s[kNT][4];
#pragma unroll
    for (int n = 0; n < kNT; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) s[n][e] = 0.f;
#pragma unroll
    for (int kk = 0; kk < 8; ++kk)
#pragma unroll
      for (int n = 0; n < kNT; n += 2) {
        uint32_t b[4];   // tokens n*8 .. +15, channels kk*16 .. +15
        ldsm4(b, kt + row_chunk(tok0 + n * 8 + (lane & 7) + ((lane >> 4) << 3), kk * 2 + ((lane >> 3) & 1)));
        mma_16816(s[n], qf[kk], b[0], b[1]);
        mma_16816(s[n + 1], qf[kk], b[2], b[3]);
      }
    // ---- masks (tiles that every row sees whole need none), running maximum
    const uint64_t mask = s_mask[st];
    const int pos0 = cur.tile * kTile;
    const bool edge = mask != ~0ull || pos0 + kTile > cur.len - p.T + 1;
    float mx[2] = {m2[0], m2[1]};
#pragma unroll
    for (int n = 0; n < kNT; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) s[n][e] *= sl2;
    if (edge) {
      const uint64_t seen[2] = {mask & first_tokens(lim[0] - pos0), mask & first_tokens(lim[1] - pos0)};
#pragma unroll
      for (int n = 0; n < kNT; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (!(seen[e >> 1] >> (tok0 + n * 8 + t4 * 2 + (e & 1)) & 1)) s[n][e] = -INFINITY;
    }
#pragma unroll
    for (int n = 0; n < kNT; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) mx[e >> 1] = fmaxf(mx[e >> 1], s[n][e]);
    float base[2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      mx[r] = fmaxf(mx[r], __shfl_xor_sync(0xffffffffu, mx[r], 1));
      mx[r] = fmaxf(mx[r], __shfl_xor_sync(0xffffffffu, mx[r], 2));
      base[r] = mx[r] == -INFINITY ? 0.f : mx[r];   // nothing seen yet: every weight is 2^-inf = 0
    }
    if (__any_sync(0xffffffffu, mx[0] != m2[0] || mx[1] != m2[1])) {
      const float c0 = fast_exp2(m2[0] - base[0]), c1 = fast_exp2(m2[1] - base[1]);
      l2[0] *= c0;
      l2[1] *= c1;
#pragma unroll
      for (int n = 0; n < 16; ++n) {
        o[n][0] *= c0; o[n][1] *= c0;
        o[n][2] *= c1; o[n][3] *= c1;
      }
      m2[0] = mx[0];
      m2[1] = mx[1];
    }
    uint32_t pf[kNT / 2][4];
#pragma unroll
    for (int n = 0; n < kNT; ++n) {
      float e0 = fast_exp2(s[n][0] - base[0]), e1 = fast_exp2(s[n][1] - base[0]);
      float e2 = fast_exp2(s[n][2] - base[1]), e3 = fast_exp2(s[n][3] - base[1]);
      l2[0] += e0 + e1;
      l2[1] += e2 + e3;
      pf[n >> 1][(n & 1) * 2] = pack_bf16x2(e0, e1);
      pf[n >> 1][(n & 1) * 2 + 1] = pack_bf16x2(e2, e3);
    }
    // ---- values
    auto value_pair = [&](uint32_t (&b)[4], int k, int n) {   // tokens k*16 .. +15, channels n*8 .. +15
      ldsm4_t(b, vt + row_chunk(tok0 + k * 16 + (lane & 15), n + (lane >> 4)));
    };
    if (!edge) {
#pragma unroll
      for (int k = 0; k < kNT / 2; ++k)
#pragma unroll
        for (int n = 0; n < 16; n += 2) {
          uint32_t b[4];
          value_pair(b, k, n);
          mma_16816(o[n], pf[k], b[0], b[1]);
          mma_16816(o[n + 1], pf[k], b[2], b[3]);
        }
    } else {
      // Rows that are not there hold anything, and NaN and infinities would survive their zero weights: they are cleared
      // on the way.  So would a new token's value row that earlier new tokens must not see: where one is not finite the
      // new tokens take their products one at a time, with the rows behind them cleared.
      const auto cleared = [&](uint32_t (&b)[4], int k, uint64_t rows) {
        const uint32_t r = static_cast<uint32_t>(rows >> (tok0 + k * 16 + 2 * t4));
        const uint32_t lo = pick2(r), hi = pick2(r >> 8);
        b[0] &= lo; b[2] &= lo;
        b[1] &= hi; b[3] &= hi;
      };
      bool bad = false;
      const uint64_t later = mask & ~first_tokens(cur.len - p.T + 1 - pos0);
      if (later) {
#pragma unroll
        for (int k = 0; k < kNT / 2; ++k)
#pragma unroll
          for (int n = 0; n < 16; n += 2) {
            uint32_t b[4];
            value_pair(b, k, n);
            cleared(b, k, later);
#pragma unroll
            for (int e = 0; e < 4; ++e) bad |= (b[e] & 0x7F80u) == 0x7F80u || (b[e] & 0x7F800000u) == 0x7F800000u;
          }
        bad = __any_sync(0xffffffffu, bad);
      }
      const int row0 = (cur.hr % p.row_blocks) * kRows + 16 * wr + g;
#pragma unroll 1
      for (int t = bad ? p.T - 1 : 0; t >= 0; --t) {
        const uint64_t rows = bad ? mask & first_tokens(cur.len - p.T + t + 1 - pos0) : mask;
        const bool on0 = !bad || row0 / p.G == t, on1 = !bad || (row0 + 8) / p.G == t;
#pragma unroll
        for (int n = 0; n < 16; n += 2) {
          float x[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
          for (int k = 0; k < kNT / 2; ++k) {
            uint32_t b[4];
            value_pair(b, k, n);
            cleared(b, k, rows);
            mma_16816(x[0], pf[k], b[0], b[1]);
            mma_16816(x[1], pf[k], b[2], b[3]);
          }
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            if (on0) { o[n + y][0] += x[y][0]; o[n + y][1] += x[y][1]; }
            if (on1) { o[n + y][2] += x[y][2]; o[n + y][3] += x[y][3]; }
          }
        }
      }
    }

    // ---- the item's (or the stretch's) end: join the warps of each row group, write the rows or the part
    const bool item_ends = cur.tile + 1 == tile_count(cur.len);
    if (item_ends || stretch_ends) {
      const bool from_start = cur.tile == i - begun;   // the item began in this stretch, too
      const bool whole = item_ends && from_start;
      float l0 = l2[0], l1 = l2[1];
      l0 += __shfl_xor_sync(0xffffffffu, l0, 1);
      l0 += __shfl_xor_sync(0xffffffffu, l0, 2);
      l1 += __shfl_xor_sync(0xffffffffu, l1, 1);
      l1 += __shfl_xor_sync(0xffffffffu, l1, 2);
      meet();   // tile i has been read: its stage takes the sums
      // (a cluster's CTA ends here: no stage is in use any more)
      float *so = reinterpret_cast<float *>(sm + (ranks > 1 ? 1 : st) * kStageBytes);
#pragma unroll
      for (int n = 0; n < 16; ++n) {
        const int c = (n * 8 + t4 * 2) ^ (g << 3);
        *reinterpret_cast<float2 *>(so + (warp * 16 + g) * kD + c) = make_float2(o[n][0], o[n][1]);
        *reinterpret_cast<float2 *>(so + (warp * 16 + g + 8) * kD + c) = make_float2(o[n][2], o[n][3]);
      }
      if (t4 == 0) {
        s_ml[(warp * 16 + g) * 2] = m2[0];
        s_ml[(warp * 16 + g) * 2 + 1] = l0;
        s_ml[(warp * 16 + g + 8) * 2] = m2[1];
        s_ml[(warp * 16 + g + 8) * 2 + 1] = l1;
      }
      meet();
      const int rb = cur.hr % p.row_blocks, h = cur.hr / p.row_blocks;
      const int slot = 2 * blockIdx.x + (from_start ? 1 : 0);
      for (int r = warp; r < kRows; r += kComputeWarps) {
        const int row = rb * kRows + r, t = row / p.G;
        if (t >= p.T) break;
        const int gr = r >> 4, rr = r & 15;
        float mm = -INFINITY;
#pragma unroll
        for (int w = 0; w < WT; ++w) mm = fmaxf(mm, s_ml[((w * WR + gr) * 16 + rr) * 2]);
        const float bs = mm == -INFINITY ? 0.f : mm;
        float ll = 0.f;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < WT; ++w) {
          const int wi = (w * WR + gr) * 16 + rr;
          const float c = fast_exp2(s_ml[wi * 2] - bs);
          const float4 x = *reinterpret_cast<const float4 *>(so + wi * kD + ((lane * 4) ^ ((rr & 7) << 3)));
          ll += c * s_ml[wi * 2 + 1];
          acc.x += c * x.x; acc.y += c * x.y; acc.z += c * x.z; acc.w += c * x.w;
        }
        if (ranks > 1) {
          *reinterpret_cast<float4 *>(sm + (r * kD + lane * 4) * 4) = acc;
          if (lane == 0) *reinterpret_cast<float2 *>(sm + OFF_CML + 8 * r) = make_float2(mm, ll);
        } else if (whole) {
          paged_store_row(p, cur.b, t, h * p.G + row % p.G, lane, acc, mm, ll);
        } else {
          float *part = p.parts + (static_cast<size_t>(slot) * kRows + r) * kPagedPartFloats;
          *reinterpret_cast<float4 *>(part + lane * 4) = acc;
          if (lane == 0) *reinterpret_cast<float2 *>(part + kD) = make_float2(mm, ll);
        }
      }
      fresh = true;
      sm100::fence_async_smem();   // (the stage's next tile comes behind these accesses)
    }
    __syncwarp();
    if (lane == 0) sm100::mbar_arrive(&freed[st]);
    if (stretch_ends) break;
  }
  __syncwarp();
  finish();
}

// Joins the parts of the items that the stretches cut.  Every CTA lists the joins (few places hold one) and takes rows of
// them in turn, with 2, 4, 8 or 16 warps a row (`split`), each with every split-th part, four of them under way together.
// Bound by the latency of three dependent loads (the list, the parts, the row), so all rows go at once where they can.
constexpr int kJoinThreads = 512, kJoinWarps = kJoinThreads / 32, kJoinCtas = 304;
static_assert(kPagedMaxCtas <= kJoinThreads, "a place a thread");
__global__ void __launch_bounds__(kJoinThreads, 2) paged_join_kernel(PagedArgs p, int rows_per_item, int places) {
  __shared__ int4 s_join[kPagedMaxCtas];
  __shared__ int s_count[kJoinWarps];
  __shared__ float4 s_acc[kJoinWarps][32];
  __shared__ float2 s_ml[kJoinWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  sm100::grid_dependency_wait();
  int4 mine = static_cast<int>(threadIdx.x) < places ? p.joins[threadIdx.x] : make_int4(0, 0, 0, 0);
  mine.w = threadIdx.x;
  const uint32_t on = __ballot_sync(0xffffffffu, mine.x != 0);
  if (lane == 0) s_count[warp] = __popc(on);
  __syncthreads();
  int joins = 0;
#pragma unroll
  for (int i = 0; i < kJoinWarps; ++i) {
    if (i == warp && mine.x != 0) s_join[joins + __popc(on & ((1u << lane) - 1))] = mine;
    joins += s_count[i];
  }
  __syncthreads();
  const int rows = min(rows_per_item, p.T * p.G);   // (a last row block may have fewer)
  const int units = joins * rows, most = gridDim.x * kJoinWarps;
  int split = kJoinWarps;
  while (split > 2 && units * split > most) split >>= 1;
  const int w = warp & (split - 1), per_cta = kJoinWarps / split;
  for (int at0 = per_cta * blockIdx.x; at0 < units; at0 += per_cta * gridDim.x) {
    const int at = at0 + warp / split;
    const int4 j = s_join[min(at, units - 1) / rows];
    const int cut = j.w, r = at % rows;
    const int rb = j.z % p.row_blocks, h = j.z / p.row_blocks;
    const int row = rb * rows_per_item + r, t = row / p.G;
    const bool there = at < units && t < p.T;
    float m = -INFINITY, l = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    if (there) {
      // part 0: the stretch before the cut, in its last slot; part n: the n-th stretch from the cut on, in its first
      auto part = [&](int n) {
        const int slot = n == 0 ? 2 * (cut - 1) + 1 : 2 * (cut + n - 1);
        return p.parts + (static_cast<size_t>(slot) * rows_per_item + r) * kPagedPartFloats;
      };
      for (int n0 = w; n0 < j.x; n0 += 4 * split) {
        float2 ml[4];
        float4 x[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int n = n0 + i * split;
          ml[i] = make_float2(-INFINITY, 0.f);
          x[i] = make_float4(0.f, 0.f, 0.f, 0.f);
          if (n < j.x) {
            const float *q = part(n);
            ml[i] = *reinterpret_cast<const float2 *>(q + kD);
            x[i] = *reinterpret_cast<const float4 *>(q + lane * 4);
          }
        }
        float top = m;
#pragma unroll
        for (int i = 0; i < 4; ++i) top = fmaxf(top, ml[i].x);
        const float base = top == -INFINITY ? 0.f : top, c0 = fast_exp2(m - base);
        l *= c0;
        acc = make_float4(c0 * acc.x, c0 * acc.y, c0 * acc.z, c0 * acc.w);
        m = top;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float c = fast_exp2(ml[i].x - base);
          l += c * ml[i].y;
          acc.x += c * x[i].x; acc.y += c * x[i].y; acc.z += c * x[i].z; acc.w += c * x[i].w;
        }
      }
      s_acc[warp][lane] = acc;
      if (lane == 0) s_ml[warp] = make_float2(m, l);
    }
    __syncthreads();
    if (there && w == 0) {
      float top = m;
      for (int i = 1; i < split; ++i) top = fmaxf(top, s_ml[warp + i].x);
      const float base = top == -INFINITY ? 0.f : top, c0 = fast_exp2(m - base);
      l *= c0;
      acc = make_float4(c0 * acc.x, c0 * acc.y, c0 * acc.z, c0 * acc.w);
      for (int i = 1; i < split; ++i) {
        const float2 ml = s_ml[warp + i];
        const float4 x = s_acc[warp + i][lane];
        const float c = fast_exp2(ml.x - base);
        l += c * ml.y;
        acc.x += c * x.x; acc.y += c * x.y; acc.z += c * x.z; acc.w += c * x.w;
      }
      paged_store_row(p, j.y, t, h * p.G + row % p.G, lane, acc, top, l);
    }
    __syncthreads();
  }
}

// Tiles for each CTA of a cluster, at most.  Measured (16 query, 2 key heads, requests of one length; cut against clusters):
// one request of 257 tokens 8.9 and 6.3 us, of 2048 11.5 and 9.9, of 4096 (8 tiles a CTA) 15.6 and 15.0; 16 of 2048 (4
// tiles) 14.5 and 11.4; 120 of 257 (5 tiles) 16.1 and 11.8, of 4096 (64 tiles) 85 and 91.  The host knows no lengths, only how
// many tokens the table's rows hold, so this is a limit on the table; a CTA takes 1.3 us a tile, and where one request is
// much longer than the others only stretches share it out.  By these figures the limit could be higher for requests of one
// length (5 tiles gain 4.3 us), and short requests in a wide table take the cut and its join all the same.
constexpr int kWholeTiles = 4;
// Boxes of fewer rows are not worth a TMA copy each (four a box).  Measured over 64 x 8192 tokens, 2 key heads: boxes of 8
// 109 us against 95 us by asynchronous copies, of 16 and more 90 to 92 us (copies by one warp instead of two: 133 us).
constexpr int kLeastBox = 16;

// false: the strides or sizes are none that a tensor map takes
bool make_page_map(CUtensorMap *map, const uint16_t *pages, int64_t page_stride, int64_t token_stride, int64_t head_stride,
                   const PagedArgs &a, int box) {
  const int64_t most = (int64_t(1) << 39) / 2;
  if (a.Hk == 1) head_stride = kD;   // (of one alone the stride may be anything)
  if (a.num_pages == 1) page_stride = kD;
  if (a.num_pages < 1 || page_stride <= 0 || token_stride <= 0 || head_stride <= 0 || page_stride >= most ||
      token_stride >= most || head_stride >= most)
    return false;
  const uint64_t dims[4] = {kD, static_cast<uint64_t>(a.Hk), static_cast<uint64_t>(a.page), static_cast<uint64_t>(a.num_pages)};
  const uint64_t strides[3] = {static_cast<uint64_t>(head_stride) * 2, static_cast<uint64_t>(token_stride) * 2,
                               static_cast<uint64_t>(page_stride) * 2};
  const uint32_t boxes[4] = {64, 1, static_cast<uint32_t>(box), 1};
  return make_bf16_map(map, pages, 4, dims, strides, boxes);
}

template <int WR>
cudaError_t launch_paged(PagedArgs a, cudaStream_t stream) {
  static std::mutex mu;
  static uint64_t done = 0;
  if (const cudaError_t e = set_attributes_once(mu, done, [] {
        cudaError_t r = cudaFuncSetAttribute(paged_attention_kernel<WR, false>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
        if (r == cudaSuccess)
          r = cudaFuncSetAttribute(paged_attention_kernel<WR, true>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
        return r;
      }))
    return e;
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    sms = 152;
  a.row_blocks = (a.T * a.G + 16 * WR - 1) / (16 * WR);
  const int64_t items = static_cast<int64_t>(a.B) * a.Hk * a.row_blocks;
  const int64_t most = items * std::max<int64_t>(1, (a.max_len + kTile - 1) / kTile);   // tiles there can be
  const int64_t ctas = std::min(2 * sms, kPagedMaxCtas);
  // Items that all run at once and are short go to a cluster each, whose CTAs join through shared memory: the scan and the
  // join kernel cost more than the tiles.
  int ranks = kMostRanks;
  while (ranks > 1 && items * ranks > ctas) ranks >>= 1;
  const bool whole = items * ranks <= ctas && most <= items * ranks * kWholeTiles;
  while (ranks > 1 && most <= items * (ranks >> 1)) ranks >>= 1;   // no more of them than tiles
  a.cluster = ranks;
  const unsigned grid = static_cast<unsigned>(whole ? items * ranks : std::min(most, ctas));
  PagedMaps maps;
  maps.box = 1;
  while (maps.box < kTile && a.page % (2 * maps.box) == 0) maps.box *= 2;
  if (maps.box < kLeastBox || !make_page_map(&maps.k, a.k, a.k_page_stride, a.k_token_stride, a.k_head_stride, a, maps.box) ||
      !make_page_map(&maps.v, a.v, a.v_page_stride, a.v_token_stride, a.v_head_stride, a, maps.box))
    maps.box = 0;
  if (whole)
    return launch_dependent_clusters(paged_attention_kernel<WR, true>, a.cluster, grid, kThreads, kSmemBytes, stream, a, maps);
  const cudaError_t e = launch_dependent(paged_attention_kernel<WR, false>, grid, kThreads, kSmemBytes, stream, a, maps);
  if (e != cudaSuccess) return e;
  return launch_dependent(paged_join_kernel, std::min(grid * 16 * WR, static_cast<unsigned>(kJoinCtas)), kJoinThreads, 0, stream, a,
                          16 * WR, static_cast<int>(grid));
}

}  // namespace

int paged_rows_per_item(int rows) { return rows <= 16 ? 16 : rows <= 32 ? 32 : 64; }

cudaError_t launch_paged_attention(const PagedArgs &a, cudaStream_t stream) {
  if (a.B <= 0) return cudaSuccess;
  switch (paged_rows_per_item(a.T * a.G)) {
    case 16: return launch_paged<1>(a, stream);
    case 32: return launch_paged<2>(a, stream);
    default: return launch_paged<4>(a, stream);
  }
}

}  // namespace kda
