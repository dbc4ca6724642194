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
// 2. Bound by the products where a prefix meets more than about 280 rows, else by HBM.  A block is 256 rows, for two groups of 256
// threads with half a row each, against tiles of 128 tokens, or 128 rows (where there are no more) of which the groups take the
// tiles in turn.  So either way a step is two S = Q K^T and two O += P V of 128 x 128 x 128, and while one group turns its S into P the tensor
// cores work for the other: with P written over S in TMEM (S, O: 4 x 128 columns) nothing of them passes through shared memory.
// Two warps issue the products, one for each group, which hand the turn to each other; two bring tiles, one the keys and one the
// values (K and V in turn, five of 32 KB, TMA boxes of as many rows as the page's size has powers of two, 8 to 64; pages without a
// factor of 8: asynchronous copies by the same two).  Steps of all blocks stand in one line of
// which each CTA takes an equal stretch; a stretch's part of a block is one piece.
// Weights are relative to a maximum that follows the scores only when 64 weights' sum says that it is far too low (2^14): then O and l
// are multiplied, which after the first tiles hardly ever happens; a weight of 2^14 is rounded to bf16 as exactly as one below 1.
// That rounding is the tensor cores' price (both operands of a product have one type, and V is the caller's bf16): independent of the
// output's own, it is as large (1.65e-3 in the norm), so a row whose weight is spread is off by 2.3e-3.  m, l and O are fp32, and l
// and lse sum the weights as they are before it.
#include <cuda.h>

#include <algorithm>
#include <climits>
#include <type_traits>

#include "kda_cache.h"
#include "kda_hybrid.cuh"

namespace kda {
namespace {

constexpr int kSoftWarps = 16;                     // two groups of eight: each four lots of 32 rows, two warps a lot with half the tokens each
constexpr int kThreads = 32 * (kSoftWarps + 4);    // and two for products, two for loads
constexpr int kTile = 128;                         // tokens
constexpr int kBlock = 256;                        // rows
constexpr int kSlots = 5;
constexpr uint32_t kTileBytes = kTile * kD * 2;
constexpr uint32_t OFF_Q = kSlots * kTileBytes;    // two tiles of 128 rows
constexpr int kRing = 8;                           // masks of tiles: the loads are at most five tiles ahead of their readers
constexpr uint32_t OFF_MASK = OFF_Q + 2 * kTileBytes;
constexpr uint32_t OFF_BAR = OFF_MASK + kRing * 16;
// landed [5], freed [5], scores [2], weights [2], sums [2], queries, cleared, drained [2], turn [2]
constexpr int kBarriers = 2 * kSlots + 12;
constexpr uint32_t OFF_ROWS = OFF_BAR + 8 * kBarriers;   // float [2][128]: what the two halves of a row tell each other
constexpr uint32_t OFF_TMEM = OFF_ROWS + 4 * 256;
constexpr uint32_t OFF_ABORT = OFF_TMEM + 4;
constexpr uint32_t kSmemBytes = OFF_ABORT + 4 + 1024;
static_assert(kSmemBytes <= 227 * 1024, "one CTA's shared memory");
constexpr int kMostCtas = 152;
constexpr int kCost = 2;                           // units of a block besides its steps': queries and sums
// Units of a stretch at least: CTAs without one leave their SM to the requests' own tokens.  (64 x 8192, with the share below: of 1, 2, 3, 4, 6
// and 8 units 33.9, 33.8, 34.0, 33.6, 31.3 and 36.6 us; 7 groups x 4 and 192 x 40000 the same with all of them.)
constexpr int kLeastUnits = 4;
// What the requests' own tokens cost on an SM, in units of the prefixes' line: a tile of 64 tokens of a key head, with an item's queries and
// end as four tiles.  As many SMs as their share of the work are theirs from the start: one kernel's start and end lie beside the other's
// work.  (7 groups x 4 / 192 x 40000: of 0, 0.1, 0.2, 0.3 and 0.5 units 68.7, 65.9, 65.3, 66.7, 70.2 / 121.4, 119.3, 120.1, 122.7, 126.0 us; 64 x
// 8192 33.3 to 33.8 with all of them.)
constexpr int kOwnTile = 64, kOwnCost = 4;
constexpr float kOwnUnits = 0.2f;
constexpr int kPieceFloats = 136;                  // a row of a piece: 128 sums, the maximum, the sum of weights, padding to 32 bytes
constexpr float kFollow = 64 * 256.f;              // half a row's weights of a tile: their sum, up to which the maximum may be too low
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
// 16 bytes, or zeros where they are not there
__device__ __forceinline__ void cp16_or_zero(uint32_t dst, const void *src, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16 : 0) : "memory");
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 ra, rb, rd;\n\tmov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %5};\n\t"
      "add.rn.f32x2 rd, ra, rb;\n\tmov.b64 {%0, %1}, rd;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
// 32 bytes, aligned
__device__ __forceinline__ void st_global32(float *to, const uint32_t *x) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(to), "r"(x[0]), "r"(x[1]), "r"(x[2]), "r"(x[3]),
               "r"(x[4]), "r"(x[5]), "r"(x[6]), "r"(x[7])
               : "memory");
}
// Among the 64 threads of two warps: a barrier, and whether any says so.
__device__ __forceinline__ void lot_sync(uint32_t id) { asm volatile("bar.sync %0, 64;" ::"r"(id) : "memory"); }
__device__ __forceinline__ bool lot_any(uint32_t id, bool x) {
  uint32_t y;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 q, %1, 0;\n\tbar.red.or.pred p, %2, 64, q;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(y)
      : "r"(static_cast<uint32_t>(x)), "r"(id)
      : "memory");
  return y != 0;
}
// One lane of the warp, in a way that the compiler knows to be one: what it issues then takes its operands from uniform registers.
__device__ __forceinline__ bool elect() {
  uint32_t on;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(on));
  return on != 0;
}
template <typename T>
__device__ __forceinline__ T uniform(T x) { return __shfl_sync(0xffffffffu, x, 0); }
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

// of numbers that are not negative (a 64-bit division costs four of 32)
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) {
  return (a | b) >> 32 ? a / b : static_cast<int64_t>(static_cast<uint32_t>(a) / static_cast<uint32_t>(b));
}

// Where a step's keys and values stand in the order of a block's tiles.  A block of more than 128 rows: K0 V0 K1 V1 ..; else the
// first keys of both groups, then one's values and next keys, the other's values and next keys, as far as each has them.
struct Order {
  bool split;
  int first, second;   // steps of the two groups, split
  __device__ Order(bool split, int tiles) : split(split), first((tiles + 1) / 2), second(tiles / 2) {}
  __device__ int steps(int s, int tiles) const { return !split ? tiles : s ? second : first; }
  __device__ int keys(int s, int j) const { return !split ? 2 * j : j == 0 ? s : 4 * j - 1 + 2 * s; }
  __device__ int values(int s, int j) const {
    return !split ? 2 * j + 1 : s == 0 ? 4 * j + (j < second ? 2 : 1) : 4 * j + (j + 1 < second || first > second ? 4 : 3);
  }
};

constexpr int kPlanThreads = 1024;
__global__ void __launch_bounds__(kPlanThreads) shared_prefix_plan_kernel(PrefixArgs p, int ctas) {
  __shared__ int4 s_group[kPlanThreads];   // first request, rows of a key head, shared tokens, the request whose table row is read
  __shared__ int64_t s_sum[2][32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  sm100::grid_dependency_wait();
  sm100::grid_launch_dependents();
  bool bad = false;
  for (int g = tid; g < p.groups; g += kPlanThreads) {
    const int from = p.group_starts[g], to = p.group_starts[g + 1];
    bad |= from < 0 || to < from || to > p.a.B || p.prefix_lens[g] < 0;
  }
  // (requests before the first group and behind the last; if the groups are none, all)
  const int from0 = p.group_starts[0], to0 = p.group_starts[p.groups];
  bad = __syncthreads_or(bad);
  if (bad && tid == 0) atomicOr(p.a.status, KDA_DEVICE_BAD_INDEX);
  int64_t left = 0;              // own tokens' tiles of this thread's requests, and what every request costs besides
  const auto count_own = [&](int b, int from) { left += (max(0, length_of(p.a, b) - from) + kOwnTile - 1) / kOwnTile + kOwnCost; };
  for (int b = tid; b < p.a.B; b += kPlanThreads)
    if (bad || b < from0 || b >= to0) {
      p.own[b] = make_int2(0, -1);
      count_own(b, 0);
    }
  int64_t units = 0, rows = 0;   // of the groups before
  for (int g0 = 0; g0 < p.groups; g0 += kPlanThreads) {
    for (int g = g0 + warp; g < min(p.groups, g0 + kPlanThreads); g += 32) {
      const int from = bad ? 0 : p.group_starts[g], to = bad ? 0 : p.group_starts[g + 1];
      int least = p.a.max_len, count = 0, first = to;
#pragma unroll 4
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
      for (int b = from + lane; b < to; b += 32) {
        p.own[b] = len > 0 && length_of(p.a, b) > 0 ? make_int2(len, g) : make_int2(0, -1);
        count_own(b, len);
      }
      if (lane == 0) s_group[g - g0] = make_int4(from, (to - from) * p.a.T * p.a.G, len, first);
    }
    __syncthreads();
    const int g = g0 + tid;
    PrefixGroup x{};
    int64_t u = 0, r = 0;
    if (g < p.groups) {
      const int4 y = s_group[tid];
      x.b0 = y.x;
      x.rows = y.y;
      x.len = y.z;
      x.tiles = (y.z + kTile - 1) / kTile;
      x.table_row = y.w;
      if (x.len > 0) {
        const Blocks z = blocks_of(x.rows, x.tiles);
        u = z.units * p.a.Hk;
        r = z.rows * p.a.Hk;
      }
    }
    int64_t ui = u, ri = r;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t a = __shfl_up_sync(0xffffffffu, ui, o), b = __shfl_up_sync(0xffffffffu, ri, o);
      if (lane >= o) {
        ui += a;
        ri += b;
      }
    }
    if (lane == 31) {
      s_sum[0][warp] = ui;
      s_sum[1][warp] = ri;
    }
    __syncthreads();
    // (as many warps as lanes)
    const int64_t wu = s_sum[0][lane], wr = s_sum[1][lane];
    int64_t su = wu, sr = wr;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t a = __shfl_up_sync(0xffffffffu, su, o), b = __shfl_up_sync(0xffffffffu, sr, o);
      if (lane >= o) {
        su += a;
        sr += b;
      }
    }
    x.unit = units + __shfl_sync(0xffffffffu, su - wu, warp) + ui - u;
    x.piece = rows + __shfl_sync(0xffffffffu, sr - wr, warp) + ri - r;
    if (g < p.groups) p.group[g] = x;
    units += __shfl_sync(0xffffffffu, su, 31);
    rows += __shfl_sync(0xffffffffu, sr, 31);
  }
  // the sum of all threads'
#pragma unroll
  for (int o = 16; o; o >>= 1) left += __shfl_xor_sync(0xffffffffu, left, o);
  __syncthreads();   // (the last sums have been read)
  if (lane == 0) s_sum[0][warp] = left;
  __syncthreads();
  if (tid == 0) {
    left = 0;
    for (int w = 0; w < kPlanThreads / 32; ++w) left += s_sum[0][w];
    const float own = kOwnUnits * p.a.Hk * ((p.a.T * p.a.G + 63) / 64) * static_cast<float>(left);
    const int share = ctas - static_cast<int>(ctas * own / (own + static_cast<float>(units) + 1.f));
    p.plan->units = units;
    p.plan->ticket = 0;
    p.plan->stretches = static_cast<int>(min((units + kLeastUnits - 1) / kLeastUnits, static_cast<int64_t>(max(share, 1))));
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
    w.h = static_cast<int>(quotient(v, y.units));
    v -= w.h * y.units;
    const int mb = static_cast<int>(min(static_cast<int64_t>(y.count - 1), quotient(v, tiles + kCost)));
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
           *weights = scores + 2, *sums = weights + 2, *queries = sums + 2, *cleared = queries + 1, *drained = cleared + 1, *turn = drained + 2;
  volatile uint32_t *s_abort = reinterpret_cast<volatile uint32_t *>(sm + OFF_ABORT);
  uint32_t *s_tmem = reinterpret_cast<uint32_t *>(sm + OFF_TMEM);
  uint4 *s_mask = reinterpret_cast<uint4 *>(sm + OFF_MASK);
  const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  uint32_t *status = p.a.status;
  if (tid == 0) {
    for (int i = 0; i < kSlots; ++i) {
      sm100::mbar_init(&landed[i], 1);
      sm100::mbar_init(&freed[i], 2);
    }
    for (int i = 0; i < 2; ++i) {
      sm100::mbar_init(&scores[i], 1);
      sm100::mbar_init(&weights[i], 8);
      sm100::mbar_init(&drained[i], 1);
      sm100::mbar_init(&turn[i], 1);
      sm100::mbar_init(&sums[i], 1);
    }
    sm100::mbar_init(queries, kSoftWarps);
    sm100::mbar_init(cleared, 1);
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
  if (warp == kSoftWarps) {
    sm100::tmem_alloc(s_tmem, 512);
    sm100::tmem_relinquish();
  }
  sm100::tc_fence_before();
  __syncthreads();
  sm100::tc_fence_after();
  const uint32_t tmem = uniform(*s_tmem);   // scores (and weights) of a group of threads at 128 s, sums at 256 + 128 s

  if (warp < kSoftWarps) {
    // ------------------------------------------------------------------ softmax: half a row a thread
    const int s = warp >> 3, hf = (warp >> 2) & 1, r = (warp & 3) * 32 + lane;
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t t_s = tmem + lanes + 128 * s, t_o = tmem + lanes + 256 + 128 * s + 64 * hf;
    const uint32_t lot = 1 + 4 * s + (warp & 3);   // the barrier of the two warps of these rows
    volatile float *told = reinterpret_cast<volatile float *>(sm + OFF_ROWS) + 128 * s + r;
    // (a negative scale's sign goes to the queries, and so does a scale of 0: masked scores are infinite before they are scaled)
    const float sl2 = (p.a.scale == 0.f ? 1.f : fabsf(p.a.scale)) * kLog2e;
    const uint32_t flip = p.a.scale < 0.f ? 0x80008000u : 0u, keep = p.a.scale == 0.f ? 0u : ~0u;
    // the larger (the sum) of what the two halves of a row have
    const auto both = [&](float x, auto join) {
      if (hf == 0) *told = x;
      lot_sync(lot);
      if (hf) *told = x = join(*told, x);
      lot_sync(lot);
      return hf ? x : *told;
    };
    uint32_t done = 0, blocks = 0;   // steps; blocks with some
    int ring = 0;         // tiles of the blocks before
    while (walk(p, w)) {
      const int row = (w.split ? 0 : 128 * s) + r;   // of the block
      const bool mine = row < w.rows;
      if (!(w.split && s)) {
        // 16 rows a warp, two at a time
        const int r0 = 16 * (warp & 7), q_row = (w.split ? 0 : 128 * s) + r0 + (lane & 15), rr = w.row0 + q_row;
        const int64_t tok = static_cast<int64_t>(w.b0) * p.a.T + rr / p.a.G;
        const int64_t at = q_row < w.rows ? tok * p.a.q_stride + (w.h * p.a.G + rr % p.a.G) * kD : -1;
        const uint32_t to = smem + OFF_Q + s * kTileBytes;
        const int chunk = lane & 15;
        uint4 x[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int64_t from = __shfl_sync(0xffffffffu, at, 2 * i + (lane >> 4));
          x[i] = from >= 0 ? *reinterpret_cast<const uint4 *>(p.a.q + from + 8 * chunk) : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i)
          asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(to + sm100::swz_offset(128, r0 + 2 * i + (lane >> 4), 8 * chunk)),
                       "r"((x[i].x ^ flip) & keep), "r"((x[i].y ^ flip) & keep), "r"((x[i].z ^ flip) & keep), "r"((x[i].w ^ flip) & keep)
                       : "memory");
        sm100::fence_async_smem();
      }
      __syncwarp();
      if (lane == 0) sm100::mbar_arrive(queries);
      const int steps = w.split ? (w.tiles + 1 - s) / 2 : w.tiles;
      float m = -INFINITY, l = 0.f;
#pragma unroll 1
      for (int j = 0; j < steps; ++j, ++done) {
        sm100::wait_or_abort(&scores[s], done & 1, s_abort, status);
        sm100::tc_fence_after();
        const uint2 mask = reinterpret_cast<const uint2 *>(&s_mask[(ring + (w.split ? 2 * j + s : j)) % kRing])[hf];
        // 64 tokens' scores, their maximum, and with weigh their weights relative to m
        uint32_t w2[32];
        float2 sum;
        const auto pass = [&](auto weigh) {
          constexpr bool kWeigh = decltype(weigh)::value;
          const float base = m == -INFINITY ? 0.f : m;   // nothing seen yet: every weight is 2^-inf = 0
          const float2 k2 = make_float2(sl2, sl2), b2 = make_float2(-base, -base);
          float top[2] = {-INFINITY, -INFINITY};
          sum = make_float2(0.f, 0.f);
          uint32_t x[2][16];
          sm100::tmem_ld16_async(t_s + 64 * hf, x[0]);
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            uint32_t *const y = x[c & 1];
            sm100::tmem_wait_ld();
            sm100::tmem_tie<16>(y);
            if (c < 3) sm100::tmem_ld16_async(t_s + 64 * hf + 16 * (c + 1), x[(c + 1) & 1]);
            if ((mask.x & mask.y) != ~0u) {
              const uint32_t word = (c < 2 ? mask.x : mask.y) >> (16 * (c & 1));
#pragma unroll
              for (int i = 0; i < 16; ++i)
                if (!(word >> i & 1)) y[i] = __float_as_uint(-INFINITY);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const float2 v = make_float2(__uint_as_float(y[2 * i]), __uint_as_float(y[2 * i + 1]));
              if constexpr (!kWeigh) {
                top[i & 1] = fmaxf(top[i & 1], fmaxf(v.x, v.y));
              } else {
                const float2 e = exp2_2(fma2(v, k2, b2));
                sum = add2(sum, e);
                w2[8 * c + i] = pack2(e);
              }
            }
          }
          return fmaxf(top[0], top[1]) * sl2;
        };
        if (j == 0) m = both(pass(std::false_type{}), [](float a, float b) { return fmaxf(a, b); });
        pass(std::true_type{});
        if (lot_any(lot, sum.x + sum.y > kFollow || m == -INFINITY)) {
          const float top = both(pass(std::false_type{}), [](float a, float b) { return fmaxf(a, b); });
          const float to = fmaxf(top, m), f = m == to ? 1.f : fast_exp2(m - to);
          l *= f;   // (the sums are complete: their products come before those of the scores)
          m = to;
#pragma unroll 1
          for (int c = 0; c < 64; c += 16) {
            float o[16];
            sm100::tmem_ld16(t_o + c, o);
#pragma unroll
            for (int i = 0; i < 16; ++i) o[i] *= f;
            sm100::tmem_st16(t_o + c, o);
          }
          pass(std::true_type{});
          lot_sync(lot);
        }
        // (weights go where scores of both halves were: both have read theirs at the barrier above)
        tmem_st32(t_s + 32 * hf, w2);
        l += sum.x + sum.y;
        sm100::tmem_wait_st();
        sm100::tc_fence_before();
        __syncwarp();
        if (lane == 0) sm100::mbar_arrive(&weights[s]);
      }
      ring += w.tiles;
      // the piece
      l = both(l, [](float a, float b) { return a + b; });
      float *to = p.pieces + (w.piece + (w.split ? s * w.rows : 0) + row) * kPieceFloats;
      if (steps > 0) {
        sm100::wait_or_abort(&sums[s], blocks++ & 1, s_abort, status);
        sm100::tc_fence_after();
      }
#pragma unroll
      for (int c = 0; c < 64; c += 32) {
        uint32_t o[32];
        if (steps > 0) {
          tmem_ld32(t_o + c, o);
          sm100::tmem_wait_ld();
          sm100::tmem_tie<32>(o);
        } else {
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] = 0;
        }
        if (mine)
#pragma unroll
          for (int i = 0; i < 32; i += 8) st_global32(to + 64 * hf + c + i, o + i);
      }
      if (mine && hf == 0) *reinterpret_cast<float2 *>(to + kD) = make_float2(m, l);
      sm100::tc_fence_before();
      named_bar_sync<15>(32 * kSoftWarps);   // (the other group's products have read the queries)
    }
  } else if (warp < kSoftWarps + 2) {
    // ------------------------------------------------------------------ products: a warp for each group
    constexpr uint32_t kIdescS = sm100::idesc_bf16(128, 128, false, false), kIdescO = sm100::idesc_bf16(128, 128, false, true);
    const int s = warp - kSoftWarps;
    const uint32_t t_s = tmem + 128 * s, t_o = tmem + 256 + 128 * s;
    uint32_t n = 0, items = 0, done = 0, turns = 0;   // tiles of the blocks before; blocks; steps; turns
    while (uniform(static_cast<int>(walk(p, w)))) {
      const bool split = uniform(static_cast<int>(w.split));
      const int tiles = uniform(w.tiles);
      const Order order(split, tiles);
      const int steps = order.steps(s, tiles);
      const uint64_t q = sm100::desc_kmajor_base(smem + OFF_Q + (split ? 0 : s) * kTileBytes);
      sm100::wait_or_abort(queries, items++ & 1, s_abort, status);
      const auto landing = [&](int x) {   // the slot of the block's x-th tile, once it is there
        const uint32_t i = n + x, slot = i % kSlots;
        sm100::wait_or_abort(&landed[slot], i / kSlots & 1, s_abort, status);
        return slot;
      };
      const auto free = [&](uint32_t slot) {   // (two arrivals: both groups', or twice the one's that alone has the tile)
        sm100::mma_commit(&freed[slot]);
        if (split) sm100::mma_commit(&freed[slot]);
      };
      // The groups' products go in turn, a sum of the last step's and the scores of the next together: then one's softmax falls
      // into the other's products.  (Issued side by side both groups wait for their products and for their softmax at once.)
#pragma unroll 1
      for (int j = 0; j <= (split ? order.first : tiles); ++j) {
        // the weights come last: all else is waited for while they are made
        const bool sum = j > 0 && j <= steps, next = j < steps;
        uint32_t k = 0, v = 0;
        if (sum) v = landing(order.values(s, j - 1));
        if (next) k = landing(order.keys(s, j));
        sm100::wait_or_abort(&turn[s], (turns++ + 1 - s) & 1, s_abort, status);   // (the first group's first is given)
        if (sum) sm100::wait_or_abort(&weights[s], done++ & 1, s_abort, status);
        if (elect()) {
          sm100::tc_fence_after();
          if (sum) {
            const uint64_t b = sm100::desc_mnmajor_base(smem + v * kTileBytes, 128);
#pragma unroll
            for (int i = 0; i < 8; ++i) sm100::mma_bf16_tmem_a(t_o, t_s + 8 * i, b + sm100::mnmajor_step(i), kIdescO, j > 1 || i > 0);
          }
          if (next) {
            const uint64_t b = sm100::desc_kmajor_base(smem + k * kTileBytes);
#pragma unroll
            for (int i = 0; i < 8; ++i) sm100::mma_bf16(t_s, q + sm100::kmajor_step(128, i), b + sm100::kmajor_step(128, i), kIdescS, i > 0);
            sm100::mma_commit(&scores[s]);
          }
          sm100::mbar_arrive(&turn[1 - s]);
          if (sum && !next) sm100::mma_commit(&sums[s]);   // (else the scores behind them say that the sums are there)
          if (sum) free(v);
          if (next) free(k);
        }
        __syncwarp();
      }
      n += 2 * tiles;
    }
    // (nothing is in flight behind this, after a timeout either)
    if (elect()) sm100::mma_commit(&drained[s]);
    __syncwarp();
    sm100::mbar_wait(&drained[s], 0);
  } else {
    // ------------------------------------------------------------------ loads: a warp for the keys, one for the values
    const bool values = warp == kSoftWarps + 3;
    const int box = maps.box, boxes = box ? kTile / box : 0, lots = box ? 1 : 4;
    const CUtensorMap *map = values ? &maps.v : &maps.k;
    const int64_t page_stride = values ? p.a.v_page_stride : p.a.k_page_stride, token_stride = values ? p.a.v_token_stride : p.a.k_token_stride;
    const int page = p.a.page, page_step = kTile / page, row_step = kTile - page_step * page;   // from a tile to the next
    uint32_t n = 0, fixes = 0, ring = 0, last = 0;   // tiles of the blocks before; cleared tiles; keys' tiles; the last one asked for
    bool any = false;
    // copies whose arrival is due, at most two
    uint32_t pending = 0, due0 = 0, due1 = 0;
    const auto arrive_copies = [&](uint32_t most) {   // of all but the last `most`
      if (pending <= most) return;
      if (most) asm volatile("cp.async.wait_group 1;" ::: "memory");
      else asm volatile("cp.async.wait_group 0;" ::: "memory");
      sm100::fence_async_smem();
      __syncwarp();
      for (; pending > most; --pending) {
        if (lane == 0) sm100::mbar_arrive(&landed[due0]);
        due0 = due1;
      }
      __syncwarp();
    };
    bool stop = false;
    while (!stop && uniform(static_cast<int>(walk(p, w)))) {
      const bool split = uniform(static_cast<int>(w.split));
      const int tiles = uniform(w.tiles), first = uniform(w.tile), len = uniform(w.len), head = uniform(w.h);
      const Order order(split, tiles);
      const int32_t *table = p.a.table + static_cast<int64_t>(w.table_row) * p.a.table_stride;
      const uint16_t *base = (values ? p.a.v : p.a.k) + head * (values ? p.a.v_head_stride : p.a.k_head_stride);
      // page (the place in the table's row) and row in it of the lane's box, or of its four tokens; ids are looked up a tile earlier
      int at[4], row[4], id[4], next[4] = {INT_MIN, INT_MIN, INT_MIN, INT_MIN};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (i >= lots) break;
        const int pos = first * kTile + (box ? lane * box : 32 * i + lane);
        at[i] = pos / page;
        row[i] = pos - at[i] * page;
      }
      const auto look = [&](int tile) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (i >= lots) break;
          const int in_tile = box ? lane * box : 32 * i + lane;
          next[i] = in_tile < kTile && tile * kTile + in_tile < len ? table[at[i]] : INT_MIN;
        }
      };
      look(first);
      for (int x = 0; x < tiles; ++x) {
        const int tile = first + x, count = min(kTile, len - tile * kTile);
        int from[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (i >= lots) break;
          id[i] = next[i];
          from[i] = row[i];
          at[i] += page_step;
          row[i] += row_step;
          if (row[i] >= page) {
            row[i] -= page;
            ++at[i];
          }
        }
        if (x + 1 < tiles) look(tile + 1);
        const int s = split ? x & 1 : 0, j = split ? x >> 1 : x;
        const uint32_t i = n + (values ? order.values(s, j) : order.keys(s, j)), slot = i % kSlots, dst = smem + slot * kTileBytes;
        uint32_t on[4] = {0, 0, 0, 0};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          if (k >= lots) break;
          const bool ok = id[k] >= 0 && id[k] < p.a.num_pages;
          if (!values && !ok && id[k] != INT_MIN) atomicOr(status, KDA_DEVICE_BAD_PAGE);
          on[k] = __ballot_sync(0xffffffffu, ok);
        }
        arrive_copies(1);   // (the one before this has to be told of: the slot may wait for its products)
        if (i >= kSlots) sm100::wait_or_abort(&freed[slot], (i / kSlots - 1) & 1, s_abort, status);
        if (__any_sync(0xffffffffu, *s_abort != 0)) {
          stop = true;
          break;
        }
        any = true;
        last = i;
        const bool full = count == kTile && (box ? on[0] == first_bits(boxes) : (on[0] & on[1] & on[2] & on[3]) == ~0u);
        if (!values) {
          if (full) {
            if (lane == 0) s_mask[ring % kRing] = make_uint4(~0u, ~0u, ~0u, ~0u);
          } else if (lane < 4) {
            uint32_t word = on[0];
            if (box) {
              word = 0;
              for (int t = 0; t < 32; t += 8)
                if (on[0] >> ((32 * lane + t) / box) & 1) word |= 0xFFu << t;
            } else {
#pragma unroll
              for (int k = 1; k < 4; ++k)
                if (lane == k) word = on[k];
            }
            reinterpret_cast<uint32_t *>(&s_mask[ring % kRing])[lane] = word & first_bits(count - 32 * lane);
          }
          ++ring;
          __syncwarp();
        }
        if (box) {
          uint64_t *bar = values && !full ? cleared : &landed[slot];
          // one lane brings all boxes: lanes that each bring their own are served one after another, 150 cycles each
          const uint32_t there = uniform(on[0]);
          if (elect()) sm100::mbar_arrive_expect_tx(bar, __popc(there) * box * 256);
          for (int k = 0; k < boxes; ++k) {
            const int pg = __shfl_sync(0xffffffffu, id[0], k), r = __shfl_sync(0xffffffffu, from[0], k);
            if ((there >> k & 1) && elect()) {
              const uint32_t to = dst + k * box * 128;
              tma_load_4d(to, map, 0, head, r, pg, bar);
              tma_load_4d(to + kTileBytes / 2, map, 64, head, r, pg, bar);
            }
            __syncwarp();
          }
          if (values && !full) {
            // weights of 0 do not hide what lies where nothing is: NaN and infinities
            sm100::wait_or_abort(cleared, fixes++ & 1, s_abort, status);
            for (int k = lane; k < kTile; k += 32)
              if (k >= count || !(there >> (k / box) & 1))
#pragma unroll
                for (int c = 0; c < 8; ++c) {
                  st_zero16(dst + k * 128 + 16 * c);
                  st_zero16(dst + kTileBytes / 2 + k * 128 + 16 * c);
                }
            sm100::fence_async_smem();
            __syncwarp();
            if (lane == 0) sm100::mbar_arrive(&landed[slot]);
            __syncwarp();
          }
        } else {
          // two rows at a time, 16 lanes each; rows that are not there are zeros (weights of 0 do not hide NaN and infinities)
          const int chunk = lane & 15, half = lane >> 4;
          const uint32_t panel = dst + (chunk >> 3) * (kTileBytes / 2) + half * 128;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const bool ok = on[k] >> lane & 1;
            const int64_t mine = ok ? id[k] * page_stride + from[k] * token_stride : -1;
#pragma unroll
            for (int r = 0; r < 32; r += 2) {
              const int64_t a = __shfl_sync(0xffffffffu, mine, r + half);
              cp16_or_zero(panel + (32 * k + r) * 128 + (((chunk ^ (r + half)) & 7) << 4), base + (a >= 0 ? a : 0) + 8 * chunk, a >= 0);
            }
          }
          asm volatile("cp.async.commit_group;" ::: "memory");
          if (pending++) due1 = slot;
          else due0 = slot;
        }
      }
      n += 2 * tiles;
    }
    arrive_copies(0);
    if (*s_abort && box && any) {   // (what was asked for lands before the CTA ends)
      for (uint32_t i = last >= kSlots ? last - kSlots + 1 : 0; i <= last; ++i) sm100::mbar_wait(&landed[i % kSlots], i / kSlots & 1);
      if (fixes) sm100::mbar_wait(cleared, (fixes - 1) & 1);
    }
    __syncwarp();
  }
  __syncthreads();
  if (warp == kSoftWarps) {
    sm100::tc_fence_after();
    sm100::tmem_dealloc(tmem, 512);
  }
}

// ---------------------------------------------------------------- the join
// The parts of a row: the pieces of its group's prefix, then its own tokens' (one, or those of the stretches that cut its item).
// 16 lanes take a row, eight channels each, four parts under way together; where rows are few, split lots of 16 lanes a row, which
// meet in shared memory.  Bound by the latency of the request, its group, the parts and the row, so as many rows as can be go at
// once.
constexpr int kJoinThreads = 256, kJoinLots = kJoinThreads / 16, kJoinCtas = 3 * kMostCtas;
__device__ __forceinline__ void add_part(float (&acc)[8], float c, const float4 (&x)[2]) {
  acc[0] += c * x[0].x; acc[1] += c * x[0].y; acc[2] += c * x[0].z; acc[3] += c * x[0].w;
  acc[4] += c * x[1].x; acc[5] += c * x[1].y; acc[6] += c * x[1].z; acc[7] += c * x[1].w;
}
__global__ void __launch_bounds__(kJoinThreads, 3) shared_prefix_join_kernel(PrefixArgs p, int rows_per_item, int split) {
  __shared__ float4 s_acc[kJoinLots][16][2];
  __shared__ float2 s_ml[kJoinLots];
  const PagedArgs &a = p.a;
  const int tid = threadIdx.x, lane = tid & 15, lot = tid >> 4;
  sm100::grid_dependency_wait();
  sm100::grid_launch_dependents();
  const int Hq = a.Hk * a.G, per_cta = kJoinLots / split, w = lot & (split - 1);
  const int64_t rows = static_cast<int64_t>(a.B) * a.T * Hq, units = p.plan->units, stretches = p.plan->stretches;
  for (int64_t at0 = static_cast<int64_t>(per_cta) * blockIdx.x; at0 < rows; at0 += static_cast<int64_t>(per_cta) * gridDim.x) {
    const int64_t at = at0 + lot / split;
    const bool there = at < rows;
    const int64_t tok = quotient(there ? at : 0, Hq);
    const int head = static_cast<int>((there ? at : 0) - tok * Hq), b = static_cast<int>(tok) / a.T, t = static_cast<int>(tok) - b * a.T;
    float m = -INFINITY, l = 0.f;
    float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (there) {
      const int2 own = p.own[b];
      const float4 end = *reinterpret_cast<const float4 *>(a.rows + at * kPagedPartFloats + kD);
      const int h = head / a.G, row = t * a.G + head - h * a.G, cut = __float_as_int(end.w);
      const int parts = paged_parts_there(__float_as_int(end.z), cut) ? __float_as_int(end.z) : 0;   // (0: the row is whole)
      // the prefix: the stretches that hold steps of the block, two pieces each where the groups of threads took its tiles in turn
      int64_t base = 0;
      int pieces = 0, twice = 1, second = 0;
      if (own.y >= 0) {
        const PrefixGroup &g = p.group[own.y];
        const Blocks y = blocks_of(g.rows, g.tiles);
        const int rr = (b - g.b0) * a.T * a.G + row, mb = rr / kBlock;
        const bool last_block = mb == y.count - 1;
        const int64_t first = g.unit + h * y.units + static_cast<int64_t>(mb) * (g.tiles + kCost) + kCost;
        const int64_t last = first + (last_block ? y.last_steps : g.tiles) - 1;
        const int c0 = static_cast<int>(quotient((first + 1) * stretches - 1, units)),
                  c1 = static_cast<int>(quotient((last + 1) * stretches - 1, units));
        twice = last_block && y.split ? 2 : 1;
        second = y.last_rows;
        pieces = (c1 - c0 + 1) * twice;
        base = g.piece + h * y.rows + mb * kBlock + static_cast<int64_t>(c0) * kBlock + rr % kBlock;
      }
      const auto part = [&](int n) -> const float * {
        if (n < pieces) {
          const int c = twice == 2 ? n >> 1 : n;
          return p.pieces + (base + static_cast<int64_t>(c) * kBlock + (twice == 2 && (n & 1) ? second : 0)) * kPieceFloats;
        }
        n -= pieces;
        if (!parts) return a.rows + at * kPagedPartFloats;
        return a.parts + (static_cast<size_t>(paged_part_slot(cut, n)) * rows_per_item + row % rows_per_item) * kPagedPartFloats;
      };
      const int count = pieces + (parts ? parts : 1);
      for (int n0 = w; n0 < count; n0 += 4 * split) {
        float2 ml[4];
        float4 x[4][2];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int n = n0 + i * split;
          ml[i] = make_float2(-INFINITY, 0.f);
          x[i][0] = x[i][1] = make_float4(0.f, 0.f, 0.f, 0.f);
          if (n < count) {
            const float *from = part(n);
            ml[i] = *reinterpret_cast<const float2 *>(from + kD);
            x[i][0] = *reinterpret_cast<const float4 *>(from + lane * 4);
            x[i][1] = *reinterpret_cast<const float4 *>(from + 64 + lane * 4);
          }
        }
        float top = m;
#pragma unroll
        for (int i = 0; i < 4; ++i) top = fmaxf(top, ml[i].x);
        const float from = top == -INFINITY ? 0.f : top, c0 = fast_exp2(m - from);
        l *= c0;
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[i] *= c0;
        m = top;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float c = fast_exp2(ml[i].x - from);
          l += c * ml[i].y;
          add_part(acc, c, x[i]);
        }
      }
      if (split > 1) {
        s_acc[lot][lane][0] = make_float4(acc[0], acc[1], acc[2], acc[3]);
        s_acc[lot][lane][1] = make_float4(acc[4], acc[5], acc[6], acc[7]);
        if (lane == 0) s_ml[lot] = make_float2(m, l);
      }
    }
    if (split > 1) __syncthreads();
    if (there && w == 0) {
      float top = m;
      for (int i = 1; i < split; ++i) top = fmaxf(top, s_ml[lot + i].x);
      const float from = top == -INFINITY ? 0.f : top, c0 = fast_exp2(m - from);
      l *= c0;
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[i] *= c0;
      for (int i = 1; i < split; ++i) {
        const float2 ml = s_ml[lot + i];
        const float c = fast_exp2(ml.x - from);
        l += c * ml.y;
        add_part(acc, c, s_acc[lot + i][lane]);
      }
      const float inv = l == 0.f ? 0.f : 1.0f / l;   // a row that sees nothing: zeros
      uint16_t *to = a.out + tok * a.out_stride + static_cast<int64_t>(head) * kD + lane * 4;
      *reinterpret_cast<uint2 *>(to) = make_uint2(pack_bf16x2(acc[0] * inv, acc[1] * inv), pack_bf16x2(acc[2] * inv, acc[3] * inv));
      *reinterpret_cast<uint2 *>(to + 64) = make_uint2(pack_bf16x2(acc[4] * inv, acc[5] * inv), pack_bf16x2(acc[6] * inv, acc[7] * inv));
      if (a.lse && lane == 0) a.lse[at] = l == 0.f ? -INFINITY : (top + log2f(l)) * 0.6931471805599453f;
    }
    if (split > 1) __syncthreads();
  }
}

// Bytes of prefixes that requests could read again, from which on they are shared.  The table's width bounds them; the host knows
// no lengths.  Measured, alone against shared (one group, own tokens to 200, tables to the longest request when alone; h: key heads): 16
// requests x 4096 tokens (2 h, 64 MB) 17.6 and 24.5 us, 192 x 256 (2 h, 96 MB) 20.6 and 28.2, 16 x 16384 (1 h, 122 MB) 23.4 and 25.3, 64 x 256 (8 h,
// 126 MB) 22.3 and 28.5, 64 x 4096 (1 h, 134 MB) 24.2 and 25.0; 4 x 16384 (8 h, 195 MB) 35.9 and 25.7, 16 x 16384 (2 h, 244 MB) 36.0 and 26.3, 192 x 1024
// (2 h, 239 MB) 34.4 and 29.9, 64 x 16384 (2 h, 1 GB) 111 and 34; where many requests share little, sharing loses beyond it, too (192 x 256, 8 h,
// 382 MB: 49.1 and 55.7).  A table wider than the requests counts as wide as it is: 4 x 500 tokens (2 h) take 8.2 us in a table of their length
// and 20.9 in one for 131072 tokens, 16 x 4096 17.3 and 24.8, 192 x 256 20.8 and 29.7, 64 x 4096 26.3 and 26.5.
constexpr int64_t kLeastAgain = 160 << 20;

}  // namespace

size_t shared_prefix_bytes(int B, int T, int Hq, int Hk, int groups, uint8_t *base, PrefixArgs *args) {
  const auto up = [](size_t n) { return (n + 255) & ~size_t(255); };
  const size_t rows = static_cast<size_t>(B) * T * Hq, row = kPagedPartFloats * sizeof(float);
  // blocks whose tiles are taken in turn have two pieces a row: one block of at most 128 rows for each group and key head
  const size_t twice = std::min(rows, static_cast<size_t>(std::min(groups, B)) * Hk * (kBlock / 2));
  const size_t sizes[] = {sizeof(PrefixPlan), static_cast<size_t>(groups) * sizeof(PrefixGroup), B * sizeof(int2), rows * row,
                          (rows + twice + static_cast<size_t>(kMostCtas) * kBlock) * kPieceFloats * sizeof(float)};
  size_t at[5], end = 0;
  for (int i = 0; i < 5; ++i) {
    at[i] = end;
    end += up(sizes[i]);
  }
  if (args) {
    args->plan = reinterpret_cast<PrefixPlan *>(base + at[0]);
    args->a.ticket = &args->plan->ticket;
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
  // Nothing is shared, or so little that the plan and the join cost more than reading it again: the bytes that the requests
  // of all groups but one each could read at most.
  const double again = static_cast<double>(args.a.B - std::min(args.groups, args.a.B)) * args.a.max_len * args.a.Hk * 4 * kD;
  if (args.groups == 0 || args.a.num_pages == 0 || again < kLeastAgain) return launch_paged_attention(args.a, stream);
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
  if (const cudaError_t e = launch_paged_own(a, stream)) return e;
  const int64_t rows = static_cast<int64_t>(a.B) * a.T * a.Hk * a.G;
  int split = kJoinLots;
  while (split > 1 && rows * split > static_cast<int64_t>(kJoinCtas) * kJoinLots) split >>= 1;
  const int64_t want = (rows * split + kJoinLots - 1) / kJoinLots;
  return launch_dependent(shared_prefix_join_kernel, static_cast<unsigned>(std::min<int64_t>(want, kJoinCtas)), kJoinThreads, 0, stream, args,
                          paged_rows_per_item(a.T * a.G), split);
}

}  // namespace kda
