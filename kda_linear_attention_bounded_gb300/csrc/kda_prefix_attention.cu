// Attention of new tokens over a paged cache for batches whose requests share prefixes: a prefix's keys and values meet the
// queries of all of its requests at once.
//
// The rows of a group's key head are its requests' new tokens times the query heads of the key head: row ((b - b0) T + t) G + g.
// Softmax over disjoint tokens joins from (m, l, o) = (max s, sum e^(s - m), sum e^(s - m) v), so
//   1. a plan (one CTA): what of each group's prefix every new token sees, and where its work stands in the line;
//   2. the prefixes: this file's tcgen05 kernel, parts (m, l, o) into the workspace;
//   3. the requests' own tokens: the paged attention's kernel from the first own token on, parts into the workspace;
//   4. the join of a row's parts, in the order of a fixed list.
// Each is a programmatic dependent of the one before.  Results do not depend on timing.
//
// 2. Bound by the products where a prefix meets more than about 280 rows, else by HBM.  A block is 256 rows, two groups of 128
// threads with a row each, against tiles of 128 tokens, or 128 rows (where there are no more) of which the groups take the tiles in
// turn.  So either way a step is two S = Q K^T and two O += P V of 128 x 128 x 128, and while one group turns its S into P the tensor
// cores work for the other: with P written over S in TMEM (S, O: 4 x 128 columns) nothing of them passes through shared memory.
// One warp issues the products, one brings tiles (K and V in turn, five of 32 KB, TMA boxes of as many rows as the page's size has
// powers of two, 8 to 64; pages without a factor of 8: asynchronous copies by two warps).  Steps of all blocks stand in one line of
// which each CTA takes an equal stretch; a stretch's part of a block is one piece.
// Weights are relative to a maximum that follows the scores only when it is 2^8 too low: then O and l are multiplied, which
// after the first tiles hardly ever happens; a weight up to 2^8 is rounded to bf16 as exactly as one below 1.
#include <cuda.h>

#include <algorithm>
#include <climits>

#include "kda_cache.h"
#include "kda_hybrid.cuh"

namespace kda {
namespace {

constexpr int kThreads = 384;                      // two groups of softmax warps, products, loads, loads (copies), spare
constexpr int kTile = 128;                         // tokens
constexpr int kBlock = 256;                        // rows
constexpr int kSlots = 5;
constexpr uint32_t kTileBytes = kTile * kD * 2;
constexpr uint32_t OFF_Q = kSlots * kTileBytes;    // two tiles of 128 rows
constexpr int kRing = 8;                           // masks of tiles: the loads are at most five tiles ahead of their readers
constexpr uint32_t OFF_MASK = OFF_Q + 2 * kTileBytes;
constexpr uint32_t OFF_BAR = OFF_MASK + kRing * 16;
// landed [5], freed [5], scores [2], weights [2], sums [2], queries, cleared, drained
constexpr int kBarriers = 2 * kSlots + 9;
constexpr uint32_t OFF_TMEM = OFF_BAR + 8 * kBarriers;
constexpr uint32_t OFF_ABORT = OFF_TMEM + 4;
constexpr uint32_t kSmemBytes = OFF_ABORT + 4 + 1024;
constexpr int kMostCtas = 152;
constexpr int kCost = 2;                           // units of a block besides its steps': queries and sums
constexpr float kFollow = 8.f;                     // powers of two that the maximum may be too low
constexpr int kLeastBox = 8;

__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t *r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]),
        "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]),
        "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]),
        "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t *r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
      "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};"
      ::"r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]),
      "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]),
      "r"(r[30]), "r"(r[31])
      : "memory");
}
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap *map, int c0, int c1, int c2, int c3, uint64_t *bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];"
      ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(sm100::smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ void cp16(uint32_t dst, const void *src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void st_zero16(uint32_t dst) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(dst), "r"(0) : "memory");
}
__device__ __forceinline__ uint32_t first_bits(int n) { return n <= 0 ? 0u : n >= 32 ? ~0u : (1u << n) - 1; }

// Tokens of request b that count (as in the paged attention: a length that is none is no length).
__device__ __forceinline__ int length_of(const PagedArgs &a, int b) {
  const int len = a.seq_lens[b];
  return len < 0 || len > a.max_len ? 0 : len;
}

// ---------------------------------------------------------------- the line of work
// A group's blocks: all but the last of a key head have 256 rows; the last takes its tiles in turn where it has 128 or less.
struct Blocks {
  int count, last_rows, last_steps;
  bool split;              // the last one's tiles are taken in turn
  int64_t units, rows;     // of a key head: in the line; of a stretch's pieces
};
__device__ __forceinline__ Blocks blocks_of(int rows, int tiles) {
  Blocks x;
  x.count = (rows + kBlock - 1) / kBlock;
  x.last_rows = rows - (x.count - 1) * kBlock;
  x.split = x.last_rows <= kBlock / 2;
  x.last_steps = x.split ? (tiles + 1) / 2 : tiles;
  x.units = static_cast<int64_t>(x.count - 1) * (tiles + kCost) + x.last_steps + kCost;
  x.rows = static_cast<int64_t>(x.count - 1) * kBlock + (x.split ? 2 : 1) * x.last_rows;
  return x;
}

constexpr int kPlanThreads = 1024;
__global__ void __launch_bounds__(kPlanThreads) shared_prefix_plan_kernel(PrefixArgs p, int ctas) {
  __shared__ int64_t s_sum[2][32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  sm100::grid_dependency_wait();
  sm100::grid_launch_dependents();
  bool bad = false;
  for (int g = tid; g < p.groups; g += kPlanThreads) {
    const int from = p.group_starts[g], to = p.group_starts[g + 1];
    bad |= from < 0 || to < from || to > p.a.B || p.prefix_lens[g] < 0;
  }
  for (int b = tid; b < p.a.B; b += kPlanThreads) p.own[b] = make_int2(0, -1);
  bad = __syncthreads_or(bad);
  if (bad && tid == 0) atomicOr(p.a.status, KDA_DEVICE_BAD_INDEX);
  for (int g = warp; g < p.groups; g += kPlanThreads / 32) {
    const int from = bad ? 0 : p.group_starts[g], to = bad ? 0 : p.group_starts[g + 1];
    int least = p.a.max_len, count = 0, first = to;
    for (int b = from + lane; b < to; b += 32) {
      const int len = length_of(p.a, b);
      if (len == 0) continue;
      least = min(least, max(0, len - p.a.T + 1));
      first = min(first, b);
      ++count;
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) {
      least = min(least, __shfl_xor_sync(0xffffffffu, least, o));
      first = min(first, __shfl_xor_sync(0xffffffffu, first, o));
      count += __shfl_xor_sync(0xffffffffu, count, o);
    }
    const int len = count < 2 ? 0 : min(least, p.prefix_lens[g]);   // (one request alone shares nothing)
    if (len > 0)
      for (int b = from + lane; b < to; b += 32)
        if (length_of(p.a, b) > 0) p.own[b] = make_int2(len, g);
    if (lane == 0) {
      PrefixGroup &x = p.group[g];
      x.b0 = from;
      x.rows = (to - from) * p.a.T * p.a.G;
      x.len = len;
      x.tiles = (len + kTile - 1) / kTile;
      x.table_row = first;
    }
  }
  __syncthreads();
  int64_t units = 0, rows = 0;   // of the groups before
  for (int g0 = 0; g0 < p.groups; g0 += kPlanThreads) {
    const int g = g0 + tid;
    int64_t u = 0, r = 0;
    if (g < p.groups && p.group[g].len > 0) {
      const Blocks x = blocks_of(p.group[g].rows, p.group[g].tiles);
      u = x.units * p.a.Hk;
      r = x.rows * p.a.Hk;
    }
    int64_t ui = u, ri = r;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t x = __shfl_up_sync(0xffffffffu, ui, o), y = __shfl_up_sync(0xffffffffu, ri, o);
      if (lane >= o) {
        ui += x;
        ri += y;
      }
    }
    __syncthreads();
    if (lane == 31) {
      s_sum[0][warp] = ui;
      s_sum[1][warp] = ri;
    }
    __syncthreads();
    int64_t ub = units + ui - u, rb = rows + ri - r;
#pragma unroll 8
    for (int w = 0; w < 32; ++w) {
      const int64_t x = s_sum[0][w], y = s_sum[1][w];
      if (w < warp) {
        ub += x;
        rb += y;
      }
      units += x;
      rows += y;
    }
    if (g < p.groups) {
      p.group[g].unit = ub;
      p.group[g].piece = rb;
    }
  }
  if (tid == 0) {
    p.plan->units = units;
    p.plan->stretches = static_cast<int>(min(units, static_cast<int64_t>(ctas)));
  }
}

// A stretch's part of a block, and the way along the stretch.
struct Walk {
  int64_t at, last;        // units
  int g;
  // the block
  int h, rows, row0, b0, table_row, len;
  int tile, tiles;         // its tiles in this stretch: the first, how many
  bool split;
  int64_t piece;           // its first row of pieces
};
__device__ __forceinline__ bool walk(const PrefixArgs &p, Walk &w) {
  while (w.at < w.last) {
    while (w.g + 1 < p.groups && p.group[w.g + 1].unit <= w.at) ++w.g;
    const PrefixGroup &x = p.group[w.g];
    const int tiles = x.tiles;
    const Blocks y = blocks_of(x.rows, tiles);
    int64_t v = w.at - x.unit;
    w.h = static_cast<int>(v / y.units);
    v -= w.h * y.units;
    const int mb = static_cast<int>(min(static_cast<int64_t>(y.count - 1), v / (tiles + kCost)));
    v -= static_cast<int64_t>(mb) * (tiles + kCost);
    const bool end = mb == y.count - 1;
    const int steps = end ? y.last_steps : tiles;
    const int64_t start = w.at - v + kCost;                    // the block's first step
    const int s0 = static_cast<int>(max(static_cast<int64_t>(0), v - kCost));
    const int s1 = static_cast<int>(min(static_cast<int64_t>(steps), w.last - start));
    w.at = start + steps;
    if (s1 <= s0) continue;                                    // (a stretch's last units, before a block's first step)
    w.split = end && y.split;
    w.rows = end ? y.last_rows : kBlock;
    w.row0 = mb * kBlock;
    w.b0 = x.b0;
    w.table_row = x.table_row;
    w.len = x.len;
    w.tile = w.split ? 2 * s0 : s0;
    w.tiles = (w.split ? min(2 * s1, tiles) : s1) - w.tile;
    w.piece = x.piece + w.h * y.rows + w.row0 + static_cast<int64_t>(blockIdx.x) * kBlock;
    return true;
  }
  return false;
}

// ---------------------------------------------------------------- the prefixes
struct PrefixMaps {
  CUtensorMap k, v;   // [page, token, head, 128], boxes of 64 channels x `box` tokens, 128-byte swizzle
  int box;            // 0: none, rows come by asynchronous copies
};

__global__ void __launch_bounds__(kThreads, 1) shared_prefix_kernel(PrefixArgs p, const __grid_constant__ PrefixMaps maps) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t *sm = smem_raw + (-sm100::smem_u32(smem_raw) & 1023u);
  const uint32_t smem = sm100::smem_u32(sm);
  uint64_t *landed = reinterpret_cast<uint64_t *>(sm + OFF_BAR), *freed = landed + kSlots, *scores = freed + kSlots,
           *weights = scores + 2, *sums = weights + 2, *queries = sums + 2, *cleared = queries + 1, *drained = cleared + 1;
  volatile uint32_t *s_abort = reinterpret_cast<volatile uint32_t *>(sm + OFF_ABORT);
  uint32_t *s_tmem = reinterpret_cast<uint32_t *>(sm + OFF_TMEM);
  uint4 *s_mask = reinterpret_cast<uint4 *>(sm + OFF_MASK);
  const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  uint32_t *status = p.a.status;
  if (tid == 0) {
    for (int i = 0; i < kSlots; ++i) {
      sm100::mbar_init(&landed[i], maps.box ? 1 : 2);
      sm100::mbar_init(&freed[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      sm100::mbar_init(&scores[i], 1);
      sm100::mbar_init(&weights[i], 128);
      sm100::mbar_init(&sums[i], 1);
    }
    sm100::mbar_init(queries, 256);
    sm100::mbar_init(cleared, 1);
    sm100::mbar_init(drained, 1);
    *s_abort = 0;
    sm100::fence_mbar_init();
    if (maps.box) {
      sm100::prefetch_tensormap(&maps.k);
      sm100::prefetch_tensormap(&maps.v);
    }
  }
  sm100::grid_dependency_wait();
  sm100::grid_launch_dependents();
  Walk w{};
  {
    const int64_t units = p.plan->units, stretches = p.plan->stretches;
    if (blockIdx.x < stretches) {
      w.at = units * blockIdx.x / stretches;
      w.last = units * (blockIdx.x + 1) / stretches;
    }
    if (w.at >= w.last) return;
    int lo = 0, hi = p.groups - 1;   // the last group that begins at or before the stretch
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (p.group[mid].unit <= w.at) lo = mid; else hi = mid - 1;
    }
    w.g = lo;
  }
  if (warp == 8) {
    sm100::tmem_alloc(s_tmem, 512);
    sm100::tmem_relinquish();
  }
  sm100::tc_fence_before();
  __syncthreads();
  sm100::tc_fence_after();
  const uint32_t tmem = *s_tmem;   // scores (and weights) of a group of threads at 128 s, sums at 256 + 128 s

  if (warp < 8) {
    // ------------------------------------------------------------------ softmax: a row a thread
    const int s = warp >> 2, r = tid & 127;
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t t_s = tmem + lanes + 128 * s, t_o = tmem + lanes + 256 + 128 * s;
    // (a negative scale's sign goes to the queries, and so does a scale of 0: masked scores are infinite before they are scaled)
    const float sl2 = (p.a.scale == 0.f ? 1.f : fabsf(p.a.scale)) * kLog2e;
    const uint32_t flip = p.a.scale < 0.f ? 0x80008000u : 0u, keep = p.a.scale == 0.f ? 0u : ~0u;
    uint32_t phase = 0;   // steps done
    int ring = 0;         // tiles of the blocks before
    while (walk(p, w)) {
      const int row = (w.split ? 0 : 128 * s) + r;   // of the block
      const bool mine = row < w.rows;
      if (!(w.split && s)) {
        const int rr = w.row0 + row;
        const int64_t tok = static_cast<int64_t>(w.b0) * p.a.T + rr / p.a.G;
        const uint16_t *src = p.a.q + tok * p.a.q_stride + (w.h * p.a.G + rr % p.a.G) * kD;
        const uint32_t to = smem + OFF_Q + s * kTileBytes;
#pragma unroll 8
        for (int c = 0; c < 16; ++c) {
          uint4 x = make_uint4(0, 0, 0, 0);
          if (mine) x = *reinterpret_cast<const uint4 *>(src + 8 * c);
          asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(to + sm100::swz_offset(128, r, 8 * c)), "r"((x.x ^ flip) & keep),
                       "r"((x.y ^ flip) & keep), "r"((x.z ^ flip) & keep), "r"((x.w ^ flip) & keep)
                       : "memory");
        }
        sm100::fence_async_smem();
      }
      sm100::mbar_arrive(queries);
      const int steps = w.split ? (w.tiles + 1 - s) / 2 : w.tiles;
      float m = -INFINITY, l = 0.f;
#pragma unroll 1
      for (int j = 0; j < steps; ++j, ++phase) {
        sm100::wait_or_abort(&scores[s], phase & 1, s_abort, status);
        sm100::tc_fence_after();
        uint32_t x[128];
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld32(t_s + 32 * c, x + 32 * c);
        const uint4 mask = s_mask[(ring + (w.split ? 2 * j + s : j)) % kRing];
        sm100::tmem_wait_ld();
        sm100::tmem_tie<128>(x);
        if ((mask.x & mask.y & mask.z & mask.w) != ~0u) {
          const uint32_t word[4] = {mask.x, mask.y, mask.z, mask.w};
#pragma unroll
          for (int c = 0; c < 128; ++c)
            if (!(word[c >> 5] >> (c & 31) & 1)) x[c] = __float_as_uint(-INFINITY);
        }
        float top[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) top[c] = __uint_as_float(x[c]);
#pragma unroll
        for (int c = 4; c < 128; c += 8)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            top[i] = fmaxf(top[i], c + 4 + i < 128 ? fmaxf(__uint_as_float(x[c + i]), __uint_as_float(x[c + 4 + i]))
                                                    : __uint_as_float(x[c + i]));
        const float high = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) * sl2;
        if (j == 0) {
          m = high;
        } else {
          const bool up = high > m + kFollow;
          if (__any_sync(0xffffffffu, up)) {
            sm100::wait_or_abort(&sums[s], (phase - 1) & 1, s_abort, status);
            sm100::tc_fence_after();
            const float to = up ? high : m, f = m == to ? 1.f : fast_exp2(m - to);
            l *= f;
            m = to;
#pragma unroll 1
            for (int c = 0; c < 128; c += 16) {
              float o[16];
              sm100::tmem_ld16(t_o + c, o);
#pragma unroll
              for (int i = 0; i < 16; ++i) o[i] *= f;
              sm100::tmem_st16(t_o + c, o);
            }
          }
        }
        const float base = m == -INFINITY ? 0.f : m;   // nothing seen yet: every weight is 2^-inf = 0
        float2 part[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
        const float2 k2 = make_float2(sl2, sl2), b2 = make_float2(-base, -base);
        uint32_t w2[64];
#pragma unroll
        for (int c = 0; c < 64; ++c) {
          const float2 e = exp2_2(fma2(make_float2(__uint_as_float(x[2 * c]), __uint_as_float(x[2 * c + 1])), k2, b2));
          part[c & 1].x += e.x;
          part[c & 1].y += e.y;
          w2[c] = pack2(e);
        }
        tmem_st32(t_s, w2);
        tmem_st32(t_s + 32, w2 + 32);
        l += (part[0].x + part[0].y) + (part[1].x + part[1].y);
        sm100::tmem_wait_st();
        sm100::tc_fence_before();
        sm100::mbar_arrive(&weights[s]);
      }
      ring += w.tiles;
      // the piece
      float *to = p.pieces + (w.piece + (w.split ? s * w.rows : 0) + row) * kPagedPartFloats;
      if (steps > 0) {
        sm100::wait_or_abort(&sums[s], (phase - 1) & 1, s_abort, status);
        sm100::tc_fence_after();
#pragma unroll 1
        for (int c = 0; c < 128; c += 32) {
          uint32_t o[32];
          tmem_ld32(t_o + c, o);
          sm100::tmem_wait_ld();
          sm100::tmem_tie<32>(o);
          if (mine)
#pragma unroll
            for (int i = 0; i < 32; i += 4)
              *reinterpret_cast<uint4 *>(to + c + i) = make_uint4(o[i], o[i + 1], o[i + 2], o[i + 3]);
        }
      } else if (mine) {
        for (int c = 0; c < 128; c += 4) *reinterpret_cast<uint4 *>(to + c) = make_uint4(0, 0, 0, 0);
      }
      if (mine) *reinterpret_cast<float2 *>(to + kD) = make_float2(m, l);
      sm100::tc_fence_before();
      named_bar_sync<1>(256);   // (the other group's products have read the queries)
    }
  } else if (warp == 8) {
    // ------------------------------------------------------------------ products
    constexpr uint32_t kIdescS = sm100::idesc_bf16(128, 128, false, false), kIdescO = sm100::idesc_bf16(128, 128, false, true);
    uint32_t n = 0, items = 0, done[2] = {0, 0};
    const auto take = [&] {   // the next tile's slot, once it is there
      const uint32_t slot = n % kSlots;
      sm100::wait_or_abort(&landed[slot], n / kSlots & 1, s_abort, status);
      ++n;
      return slot;
    };
    while (walk(p, w)) {
      sm100::wait_or_abort(queries, items++ & 1, s_abort, status);
      const int steps[2] = {w.split ? (w.tiles + 1) / 2 : w.tiles, w.split ? w.tiles / 2 : w.tiles};
      const auto product_s = [&](int s, uint32_t slot) {
        if (lane == 0) {
          sm100::tc_fence_after();
          const uint64_t a = sm100::desc_kmajor_base(smem + OFF_Q + (w.split ? 0 : s) * kTileBytes),
                         b = sm100::desc_kmajor_base(smem + slot * kTileBytes);
#pragma unroll
          for (int k = 0; k < 8; ++k)
            sm100::mma_bf16(tmem + 128 * s, a + sm100::kmajor_step(128, k), b + sm100::kmajor_step(128, k), kIdescS, k > 0);
          sm100::mma_commit(&scores[s]);
          if (w.split || s) sm100::mma_commit(&freed[slot]);
        }
        __syncwarp();
      };
      const auto product_o = [&](int s, uint32_t slot, bool more) {
        if (lane == 0) {
          sm100::tc_fence_after();
          const uint64_t b = sm100::desc_mnmajor_base(smem + slot * kTileBytes, 128);
#pragma unroll
          for (int k = 0; k < 8; ++k)
            sm100::mma_bf16_tmem_a(tmem + 256 + 128 * s, tmem + 128 * s + 8 * k, b + sm100::mnmajor_step(k), kIdescO, more || k > 0);
          sm100::mma_commit(&sums[s]);
          if (w.split || s) sm100::mma_commit(&freed[slot]);
        }
        __syncwarp();
      };
      uint32_t k = take(), v = 0;
      product_s(0, k);
      if (steps[1] > 0) {
        if (w.split) k = take();
        product_s(1, k);
      }
#pragma unroll 1
      for (int j = 0; j < steps[0]; ++j) {
        sm100::wait_or_abort(&weights[0], done[0]++ & 1, s_abort, status);
        v = take();
        product_o(0, v, j > 0);
        if (j + 1 < steps[0]) {
          k = take();
          product_s(0, k);
        }
        if (j < steps[1]) {
          sm100::wait_or_abort(&weights[1], done[1]++ & 1, s_abort, status);
          if (w.split) v = take();
          product_o(1, v, j > 0);
          if (j + 1 < steps[1]) {
            if (w.split) k = take();
            product_s(1, k);
          }
        }
      }
    }
    // (nothing is in flight behind this, after a timeout either)
    if (lane == 0) sm100::mma_commit(drained);
    __syncwarp();
    sm100::mbar_wait(drained, 0);
  } else if (warp == 9 || (warp == 10 && !maps.box)) {
    // ------------------------------------------------------------------ loads
    const int half = warp - 9, box = maps.box;
    uint32_t n = 0, fixes = 0, ring = 0;
    uint32_t pending = 0;   // copies whose arrival is due, at most two
    const auto arrive_copies = [&](uint32_t most) {   // of all but the last `most`
      if (pending <= most) return;
      if (most) asm volatile("cp.async.wait_group 2;" ::: "memory");
      else asm volatile("cp.async.wait_group 0;" ::: "memory");
      sm100::fence_async_smem();
      __syncwarp();
      for (; pending > most; --pending)
        if (lane == 0) sm100::mbar_arrive(&landed[(n - pending) % kSlots]);
      __syncwarp();
    };
    struct Ids {
      int id[2];          // pages of the lane's box (TMA) or of its two rows
      int tile;
    };
    const auto ask = [&](int tile) {
      Ids x;
      x.tile = tile;
      const int32_t *row = p.a.table + static_cast<int64_t>(w.table_row) * p.a.table_stride;
      if (box) {
        const int pos = tile * kTile + lane * box;
        x.id[0] = lane * box < kTile && pos < w.len ? row[pos / p.a.page] : INT_MIN;
        x.id[1] = INT_MIN;
      } else {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int pos = tile * kTile + 64 * half + 32 * i + lane;
          x.id[i] = pos < w.len ? row[pos / p.a.page] : INT_MIN;
        }
      }
      return x;
    };
    bool stop = false;
    const auto load = [&](const Ids &x, bool values) {
      if (stop) return;
      const uint32_t slot = n % kSlots, dst = smem + slot * kTileBytes;
      const int pos0 = x.tile * kTile, count = min(kTile, w.len - pos0);
      const bool ok0 = x.id[0] >= 0 && x.id[0] < p.a.num_pages, ok1 = x.id[1] >= 0 && x.id[1] < p.a.num_pages;
      if (!values && ((x.id[0] != INT_MIN && !ok0) || (x.id[1] != INT_MIN && !ok1))) atomicOr(status, KDA_DEVICE_BAD_PAGE);
      const uint32_t on0 = __ballot_sync(0xffffffffu, ok0), on1 = __ballot_sync(0xffffffffu, ok1);
      if (n >= kSlots) sm100::wait_or_abort(&freed[slot], (n / kSlots - 1) & 1, s_abort, status);
      if (__any_sync(0xffffffffu, *s_abort != 0)) {
        stop = true;
        return;
      }
      if (box) {
        const int boxes = kTile / box;
        const bool full = on0 == first_bits(boxes) && count == kTile;
        if (!values && lane < 4) {
          uint32_t word = 0;
          for (int t = 0; t < 32; t += 8)
            if (on0 >> ((32 * lane + t) / box) & 1) word |= 0xFFu << t;
          reinterpret_cast<uint32_t *>(&s_mask[ring % kRing])[lane] = word & first_bits(count - 32 * lane);
        }
        __syncwarp();
        uint64_t *bar = values && !full ? cleared : &landed[slot];
        if (lane == 0) sm100::mbar_arrive_expect_tx(bar, __popc(on0) * box * 256);
        __syncwarp();
        if (ok0) {
          const CUtensorMap *map = values ? &maps.v : &maps.k;
          const int tok = (pos0 + lane * box) % p.a.page;
          const uint32_t to = dst + lane * box * 128;
          tma_load_4d(to, map, 0, w.h, tok, x.id[0], bar);
          tma_load_4d(to + kTileBytes / 2, map, 64, w.h, tok, x.id[0], bar);
        }
        __syncwarp();
        if (bar == cleared) {
          // weights of 0 do not hide what lies where nothing is: NaN and infinities
          sm100::wait_or_abort(cleared, fixes++ & 1, s_abort, status);
          for (int row = lane; row < kTile; row += 32)
            if (row >= count || !(on0 >> (row / box) & 1))
#pragma unroll
              for (int c = 0; c < 8; ++c) {
                st_zero16(dst + row * 128 + 16 * c);
                st_zero16(dst + kTileBytes / 2 + row * 128 + 16 * c);
              }
          sm100::fence_async_smem();
          __syncwarp();
          if (lane == 0) sm100::mbar_arrive(&landed[slot]);
          __syncwarp();
        }
      } else {
        if (!values && lane < 2)
          reinterpret_cast<uint32_t *>(&s_mask[ring % kRing])[2 * half + lane] = lane ? on1 : on0;
        const int64_t ps = values ? p.a.v_page_stride : p.a.k_page_stride, ts = values ? p.a.v_token_stride : p.a.k_token_stride;
        const uint16_t *base = (values ? p.a.v : p.a.k) + w.h * (values ? p.a.v_head_stride : p.a.k_head_stride);
        const int chunk = lane & 15;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const bool ok = i ? ok1 : ok0;
          const int64_t tok = (pos0 + 64 * half + 32 * i + lane) % p.a.page;
          const int64_t at = ok ? x.id[i] * ps + tok * ts : -1;
#pragma unroll 4
          for (int r = 0; r < 32; r += 2) {
            const int from = r + (lane >> 4), row = 64 * half + 32 * i + from;
            const int64_t a = __shfl_sync(0xffffffffu, at, from);
            const uint32_t to = dst + (chunk >> 3) * (kTileBytes / 2) + row * 128 + (((chunk ^ row) & 7) << 4);
            if (a >= 0) cp16(to, base + a + 8 * chunk);
            else if (values) st_zero16(to);
          }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
      }
      ++n;
      if (!box) {
        ++pending;
        arrive_copies(2);
      }
      if (!values) ++ring;
    };
    while (!stop && walk(p, w)) {
      if (!w.split) {
        Ids x = ask(w.tile);
        for (int j = 0; j < w.tiles; ++j) {
          load(x, false);
          const Ids next = j + 1 < w.tiles ? ask(w.tile + j + 1) : x;
          load(x, true);
          x = next;
        }
      } else {
        // as the products take them: keys of both groups, then a group's values and its next keys in turn
        Ids x = ask(w.tile), y = w.tiles > 1 ? ask(w.tile + 1) : x;
        load(x, false);
        if (w.tiles > 1) load(y, false);
        for (int j = 0; j < w.tiles; j += 2) {
          const Ids x2 = j + 2 < w.tiles ? ask(w.tile + j + 2) : x, y2 = j + 3 < w.tiles ? ask(w.tile + j + 3) : y;
          load(x, true);
          if (j + 2 < w.tiles) load(x2, false);
          if (j + 1 < w.tiles) load(y, true);
          if (j + 3 < w.tiles) load(y2, false);
          x = x2;
          y = y2;
        }
      }
    }
    arrive_copies(0);
    asm volatile("cp.async.wait_all;" ::: "memory");
    if (*s_abort && box) {   // (what was asked for lands before the CTA ends)
      for (uint32_t i = n > kSlots ? n - kSlots : 0; i < n; ++i) sm100::mbar_wait(&landed[i % kSlots], i / kSlots & 1);
      if (fixes) sm100::mbar_wait(cleared, (fixes - 1) & 1);
    }
    __syncwarp();
  }
  __syncthreads();
  if (warp == 8) {
    sm100::tc_fence_after();
    sm100::tmem_dealloc(tmem, 512);
  }
}

// ---------------------------------------------------------------- the join
// The parts of a row: its own tokens' (one, or those of the stretches that cut its item), and the pieces of its group's prefix.
// split warps take a row's parts in turn, four under way together, and meet in shared memory.
constexpr int kJoinThreads = 512, kJoinWarps = kJoinThreads / 32, kJoinCtas = 304;
static_assert(kPagedMaxCtas <= kJoinThreads, "a place a thread");
__global__ void __launch_bounds__(kJoinThreads, 2) shared_prefix_join_kernel(PrefixArgs p, int rows_per_item, int row_blocks, int places,
                                                                             int split) {
  __shared__ int4 s_join[kPagedMaxCtas];
  __shared__ int s_count[kJoinWarps];
  __shared__ float4 s_acc[kJoinWarps][32];
  __shared__ float2 s_ml[kJoinWarps];
  const PagedArgs &a = p.a;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  sm100::grid_dependency_wait();
  sm100::grid_launch_dependents();
  int4 cut = static_cast<int>(threadIdx.x) < places ? a.joins[threadIdx.x] : make_int4(0, 0, 0, 0);
  cut.w = threadIdx.x;
  const uint32_t on = __ballot_sync(0xffffffffu, cut.x != 0);
  if (lane == 0) s_count[warp] = __popc(on);
  __syncthreads();
  int joins = 0;
#pragma unroll
  for (int i = 0; i < kJoinWarps; ++i) {
    if (i == warp && cut.x != 0) s_join[joins + __popc(on & ((1u << lane) - 1))] = cut;
    joins += s_count[i];
  }
  __syncthreads();
  const int Hq = a.Hk * a.G;
  const int64_t rows = static_cast<int64_t>(a.B) * a.T * Hq, units = p.plan->units, stretches = p.plan->stretches;
  const int per_cta = kJoinWarps / split, w = warp & (split - 1);
  for (int64_t at0 = static_cast<int64_t>(per_cta) * blockIdx.x; at0 < rows; at0 += static_cast<int64_t>(per_cta) * gridDim.x) {
    const int64_t at = at0 + warp / split;
    const bool there = at < rows;
    float m = -INFINITY, l = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    const int64_t tok = at / Hq;
    const int head = static_cast<int>(at - tok * Hq), b = static_cast<int>(tok / a.T), t = static_cast<int>(tok - static_cast<int64_t>(b) * a.T);
    if (there) {
      const int h = head / a.G, row = t * a.G + head % a.G;
      const int2 own = p.own[b];
      // own tokens: the item's stretches, if it was cut
      const int hr = h * row_blocks + row / rows_per_item, r = row % rows_per_item;
      int4 j = make_int4(0, 0, 0, 0);
      for (int i0 = 0; i0 < joins; i0 += 32) {
        const int4 x = i0 + lane < joins ? s_join[i0 + lane] : make_int4(0, -1, 0, 0);
        const uint32_t hit = __ballot_sync(0xffffffffu, x.y == b && x.z == hr);
        if (hit) j = s_join[i0 + __ffs(hit) - 1];
      }
      const int mine = j.x ? j.x : 1;
      // the prefix: the stretches that hold steps of the block, two pieces each where the groups of threads took its tiles in turn
      int64_t base = 0;
      int pieces = 0, twice = 1, second = 0;
      if (own.y >= 0) {
        const PrefixGroup &g = p.group[own.y];
        const Blocks y = blocks_of(g.rows, g.tiles);
        const int rr = static_cast<int>((tok - static_cast<int64_t>(g.b0) * a.T) * a.G) + head % a.G, mb = rr / kBlock;
        const bool end = mb == y.count - 1;
        const int64_t first = g.unit + h * y.units + static_cast<int64_t>(mb) * (g.tiles + kCost) + kCost;
        const int64_t last = first + (end ? y.last_steps : g.tiles) - 1;
        const int c0 = static_cast<int>(((first + 1) * stretches - 1) / units), c1 = static_cast<int>(((last + 1) * stretches - 1) / units);
        twice = end && y.split ? 2 : 1;
        second = y.last_rows;
        pieces = (c1 - c0 + 1) * twice;
        base = g.piece + h * y.rows + mb * kBlock + static_cast<int64_t>(c0) * kBlock + rr % kBlock;
      }
      const auto part = [&](int n) -> const float * {
        if (n < pieces) {
          const int c = twice == 2 ? n >> 1 : n;
          return p.pieces + (base + static_cast<int64_t>(c) * kBlock + (twice == 2 && (n & 1) ? second : 0)) * kPagedPartFloats;
        }
        n -= pieces;
        if (!j.x) return a.rows + at * kPagedPartFloats;
        // part 0: the stretch before the cut, in its last slot; part n: the n-th stretch from the cut on, in its first
        const int slot = n == 0 ? 2 * (j.w - 1) + 1 : 2 * (j.w + n - 1);
        return a.parts + (static_cast<size_t>(slot) * rows_per_item + r) * kPagedPartFloats;
      };
      const int count = pieces + mine;
      for (int n0 = w; n0 < count; n0 += 4 * split) {
        float2 ml[4];
        float4 x[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int n = n0 + i * split;
          ml[i] = make_float2(-INFINITY, 0.f);
          x[i] = make_float4(0.f, 0.f, 0.f, 0.f);
          if (n < count) {
            const float *q = part(n);
            ml[i] = *reinterpret_cast<const float2 *>(q + kD);
            x[i] = *reinterpret_cast<const float4 *>(q + lane * 4);
          }
        }
        float top = m;
#pragma unroll
        for (int i = 0; i < 4; ++i) top = fmaxf(top, ml[i].x);
        const float from = top == -INFINITY ? 0.f : top, c0 = fast_exp2(m - from);
        l *= c0;
        acc = make_float4(c0 * acc.x, c0 * acc.y, c0 * acc.z, c0 * acc.w);
        m = top;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float c = fast_exp2(ml[i].x - from);
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
      const float from = top == -INFINITY ? 0.f : top, c0 = fast_exp2(m - from);
      l *= c0;
      acc = make_float4(c0 * acc.x, c0 * acc.y, c0 * acc.z, c0 * acc.w);
      for (int i = 1; i < split; ++i) {
        const float2 ml = s_ml[warp + i];
        const float4 x = s_acc[warp + i][lane];
        const float c = fast_exp2(ml.x - from);
        l += c * ml.y;
        acc.x += c * x.x; acc.y += c * x.y; acc.z += c * x.z; acc.w += c * x.w;
      }
      const float inv = l == 0.f ? 0.f : 1.0f / l;   // a row that sees nothing: zeros
      *reinterpret_cast<uint2 *>(a.out + tok * a.out_stride + static_cast<int64_t>(head) * kD + lane * 4) =
          make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
      if (a.lse && lane == 0) a.lse[at] = l == 0.f ? -INFINITY : (top + log2f(l)) * 0.6931471805599453f;
    }
    __syncthreads();
  }
}

}  // namespace

size_t shared_prefix_bytes(int B, int T, int Hq, int Hk, int groups, uint8_t *base, PrefixArgs *args) {
  const auto up = [](size_t n) { return (n + 255) & ~size_t(255); };
  const size_t rows = static_cast<size_t>(B) * T * Hq, row = kPagedPartFloats * sizeof(float);
  // blocks whose tiles are taken in turn have two pieces a row: one block of at most 128 rows for each group and key head
  const size_t twice = std::min(rows, static_cast<size_t>(std::min(groups, B)) * Hk * (kBlock / 2));
  const size_t sizes[] = {sizeof(PrefixPlan), static_cast<size_t>(groups) * sizeof(PrefixGroup), B * sizeof(int2), rows * row,
                          (rows + twice + static_cast<size_t>(kMostCtas) * kBlock) * row};
  size_t at[5], end = 0;
  for (int i = 0; i < 5; ++i) {
    at[i] = end;
    end += up(sizes[i]);
  }
  if (args) {
    args->plan = reinterpret_cast<PrefixPlan *>(base + at[0]);
    args->group = reinterpret_cast<PrefixGroup *>(base + at[1]);
    args->own = reinterpret_cast<int2 *>(base + at[2]);
    args->a.own = args->own;
    args->a.rows = reinterpret_cast<float *>(base + at[3]);
    args->pieces = reinterpret_cast<float *>(base + at[4]);
  }
  return end;
}

cudaError_t launch_shared_prefix(const PrefixArgs &args, cudaStream_t stream) {
  if (args.a.B <= 0) return cudaSuccess;
  if (args.groups == 0 || args.a.B == 1 || args.a.num_pages == 0) return launch_paged_attention(args.a, stream);   // nothing is shared
  static std::mutex mu;
  static uint64_t done = 0;
  if (const cudaError_t e = set_attributes_once(mu, done, [] {
        return cudaFuncSetAttribute(shared_prefix_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
      }))
    return e;
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    sms = kMostCtas;
  const PagedArgs &a = args.a;
  const int ctas = std::min(sms, kMostCtas);
  if (const cudaError_t e = launch_dependent(shared_prefix_plan_kernel, 1, kPlanThreads, 0, stream, args, ctas)) return e;
  PrefixMaps maps;
  maps.box = 1;
  while (maps.box < 64 && a.page % (2 * maps.box) == 0) maps.box *= 2;
  if (maps.box < kLeastBox || !make_page_map(&maps.k, a.k, a.k_page_stride, a.k_token_stride, a.k_head_stride, a, maps.box) ||
      !make_page_map(&maps.v, a.v, a.v_page_stride, a.v_token_stride, a.v_head_stride, a, maps.box))
    maps.box = 0;
  if (const cudaError_t e = launch_dependent(shared_prefix_kernel, ctas, kThreads, kSmemBytes, stream, args, maps)) return e;
  int places = 0;
  if (const cudaError_t e = launch_paged_own(a, &places, stream)) return e;
  const int64_t rows = static_cast<int64_t>(a.B) * a.T * a.Hk * a.G;
  int split = kJoinWarps;
  while (split > 2 && rows * split > static_cast<int64_t>(kJoinCtas) * kJoinWarps) split >>= 1;
  const int64_t want = (rows * split + kJoinWarps - 1) / kJoinWarps;
  const int per = paged_rows_per_item(a.T * a.G);
  return launch_dependent(shared_prefix_join_kernel, static_cast<unsigned>(std::min<int64_t>(want, kJoinCtas)), kJoinThreads, 0, stream, args,
                          per, (a.T * a.G + per - 1) / per, places, split);
}

}  // namespace kda
