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
// SM, a fixed grid) takes an equal stretch, whatever the lengths are.  A stretch that begins or ends inside an item
// leaves its part (m, l, o) in the workspace; a second kernel, launched as a programmatic dependent, joins an item's
// parts in the order of its tokens, so results do not depend on timing.
//
// Tiles come through three 32 KB stages of 16-byte asynchronous copies (any page size and strides; page ids are
// looked up a tile earlier), rows swizzled for ldmatrix.  A CTA's rows (16, 32 or 64 of them: query heads of the key
// head x new tokens) share every key and value; with 16 rows the four warps split a tile's tokens, with 64 its rows.
// Products are mma.sync m16n8k16 (bf16, fp32 sums): even 64 rows need 64 operations per byte, which it sustains at
// HBM speed.  e^(s - m) is rounded to bf16 for the second product (the cache's own precision), l sums the unrounded.
#include <algorithm>

#include "kda_common.cuh"
#include "kda_internal.h"
#include "kda_sm100.cuh"

namespace kda {
namespace {

constexpr int kThreads = 128;
constexpr int kTile = 64;        // tokens per tile
constexpr int kStages = 3;
constexpr uint32_t kStageBytes = 2 * kTile * kD * 2;   // K rows, then V rows
constexpr uint32_t OFF_ROW = kStages * kStageBytes;    // [2][64]: element offsets of a tile's key and value rows (-1: none)
constexpr uint32_t OFF_MASK = OFF_ROW + 2 * kTile * 16; // uint32 [4][2]: which tokens of a tile are there
constexpr uint32_t OFF_ML = OFF_MASK + 32;              // float [4 warps][16 rows][2]
constexpr uint32_t OFF_SCAN = OFF_ML + 512;
constexpr uint32_t kSmemBytes = OFF_SCAN + 64;
static_assert(4 * 16 * kD * 4 <= kStageBytes, "the warps' sums fit one stage");

__device__ __forceinline__ uint32_t row_chunk(int row, int chunk) { return row * 256 + ((chunk ^ (row & 7)) << 4); }

__device__ __forceinline__ void cp16(uint32_t dst, const void *src, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16 : 0) : "memory");
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
};

// Tokens of request b; a length that is none, or that its table row cannot hold, counts as 0.
__device__ __forceinline__ int request_len(const PagedArgs &p, int b) {
  const int len = p.seq_lens[b];
  if (len < 0 || len > p.max_len) {
    if (threadIdx.x == 0) atomicOr(p.status, KDA_DEVICE_BAD_COUNT);
    return 0;
  }
  return len;
}
// Tiles of an item: an empty request keeps one (its rows are written as empty)
__device__ __forceinline__ int tile_count(int len) { return max(1, (len + kTile - 1) / kTile); }

__device__ __forceinline__ void advance(const PagedArgs &p, Cursor &c, int items_per_request) {
  if (++c.tile < c.ntiles) return;
  c.tile = 0;
  if (++c.hr < items_per_request) return;
  c.hr = 0;
  if (++c.b < p.B) {
    c.len = request_len(p, c.b);
    c.ntiles = tile_count(c.len);
  }
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

template <int WR>   // row groups of 16; the other 4 / WR warps of a row group split the tile's tokens
__global__ void __launch_bounds__(kThreads, 2) paged_attention_kernel(PagedArgs p) {
  constexpr int WT = 4 / WR, kTok = kTile / WT, kNT = kTok / 8;
  constexpr int kRows = 16 * WR;
  extern __shared__ __align__(128) uint8_t sm[];
  longlong2 *s_row = reinterpret_cast<longlong2 *>(sm + OFF_ROW);
  uint32_t *s_mask = reinterpret_cast<uint32_t *>(sm + OFF_MASK);
  float *s_ml = reinterpret_cast<float *>(sm + OFF_ML);
  const uint32_t smem = sm100::smem_u32(sm);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int wr = warp % WR, wt = warp / WR;
  const int ipr = p.Hk * p.row_blocks;   // items per request
  sm100::grid_launch_dependents();

  // ---- this CTA's stretch of the line of tiles
  int64_t *s_scan = reinterpret_cast<int64_t *>(sm + OFF_SCAN);   // [4] warp sums, then the start's request
  int64_t first = 0, last = 0, total = 0;
  int stretches;   // CTAs with tiles: every one of them has at least one
  Cursor cur;
  {
    const int per = (p.B + kThreads - 1) / kThreads;
    const int b0 = min(p.B, tid * per), b1 = min(p.B, b0 + per);
    int64_t sum = 0;
    for (int b = b0; b < b1; ++b) sum += tile_count(request_len(p, b));
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
    for (int w = 0; w < 4; ++w) {
      if (w < warp) before += s_scan[w];
      total += s_scan[w];
    }
    total *= ipr;
    before *= ipr;
    stretches = static_cast<int>(min(total, static_cast<int64_t>(gridDim.x)));
    if (blockIdx.x < stretches) {
      first = total * blockIdx.x / stretches;
      last = total * (blockIdx.x + 1) / stretches;
    }
    // the thread whose requests hold the first tile walks to it
    if (first < last && first >= before && first < before + sum * ipr) {
      int b = b0;
      int64_t at = before;
      while (true) {
        const int64_t n = static_cast<int64_t>(tile_count(request_len(p, b))) * ipr;
        if (first < at + n) break;
        at += n;
        ++b;
      }
      s_scan[4] = b;
      s_scan[5] = first - at;
    }
    __syncthreads();
  }
  if (first >= last) {
    if (tid == 0 && p.joins) p.joins[blockIdx.x] = make_int4(0, 0, 0, 0);
    return;
  }
  cur.b = static_cast<int>(s_scan[4]);
  cur.len = request_len(p, cur.b);
  cur.ntiles = tile_count(cur.len);
  cur.hr = static_cast<int>(s_scan[5] / cur.ntiles);
  cur.tile = static_cast<int>(s_scan[5] - static_cast<int64_t>(cur.hr) * cur.ntiles);
  const int ntiles_here = static_cast<int>(last - first);
  // an item that an earlier CTA began: the CTA at the first cut inside it describes the join
  if (tid == 0 && p.joins) {
    int4 j = make_int4(0, 0, 0, 0);
    if (cur.tile > 0) {
      const int64_t begin = first - cur.tile, end = begin + cur.ntiles;   // the item's tiles in the line
      if (total * (blockIdx.x - 1) / stretches <= begin) {
        int n = 1;   // stretches behind the first that begin before the item's end
        while (blockIdx.x + n < stretches && total * (blockIdx.x + n) / stretches < end) ++n;
        j = make_int4(n + 1, cur.b, cur.hr, 0);
      }
    }
    p.joins[blockIdx.x] = j;
  }

  // ---- loads: tile i of the stretch at the cursor `ld` (three tiles ahead of the products)
  Cursor ld = cur;
  int loaded = 0;   // tiles whose page ids have been asked for
  int id = 0;       // threads 0..63: the page of token `tid` of that tile
  int id_pos = 0;
  bool id_there = false;
  int id_h = 0;
  auto ask = [&] {
    id_there = false;
    if (loaded < ntiles_here) {
      if (tid < kTile) {
        id_pos = ld.tile * kTile + tid;
        id_h = ld.hr / p.row_blocks;
        if (id_pos < ld.len) {
          id = p.table[static_cast<int64_t>(ld.b) * p.table_stride + id_pos / p.page];
          id_there = true;
        }
      }
      advance(p, ld, ipr);
    }
    ++loaded;
  };
  auto place = [&] {   // the rows of tile `loaded - 1` (asked for last)
    const int i = loaded - 1;
    if (tid < kTile) {
      bool ok = id_there;
      if (ok && (id < 0 || id >= p.num_pages)) {
        atomicOr(p.status, KDA_DEVICE_BAD_PAGE);
        ok = false;
      }
      const int64_t pg = ok ? id : 0, tok = id_pos % p.page;
      s_row[(i & 1) * kTile + tid] =
          ok ? make_longlong2(pg * p.k_page_stride + tok * p.k_token_stride + id_h * p.k_head_stride,
                              pg * p.v_page_stride + tok * p.v_token_stride + id_h * p.v_head_stride)
             : make_longlong2(-1, -1);
      const uint32_t m = __ballot_sync(0xffffffffu, ok);
      if (lane == 0) s_mask[(i & 3) * 2 + warp] = m;
    }
  };
  const int lrow = tid >> 4, lchunk = tid & 15;
  auto load = [&](int i) {
    if (i < ntiles_here) {
      const uint32_t st = smem + (i % kStages) * kStageBytes;
#pragma unroll
      for (int r = 0; r < kTile; r += 8) {
        const longlong2 at = s_row[(i & 1) * kTile + r + lrow];
        const bool there = at.x >= 0;
        const uint16_t *ks = p.k + (there ? at.x : 0), *vs = p.v + (there ? at.y : 0);
        cp16(st + row_chunk(r + lrow, lchunk), ks + lchunk * 8, there);
        cp16(st + kTile * 256 + row_chunk(r + lrow, lchunk), vs + lchunk * 8, there);
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  ask(); place();
  __syncthreads();
  load(0);
  ask(); place();
  __syncthreads();
  load(1);
  ask(); place();   // tile 2's rows: read behind the first barrier of the loop

  const float sl2 = p.scale * kLog2e;
  uint32_t qf[8][4];
  float o[16][4], m2[2], l2[2];   // rows g and g + 8 of the warp's group
  int lim[2];                     // tokens each row sees
  const int g = lane >> 2, t4 = lane & 3;
  bool fresh = true;              // an item begins

  for (int i = 0; i < ntiles_here; ++i) {
    asm volatile("cp.async.wait_group 1;" ::: "memory");
    __syncthreads();   // tile i has landed; tile i - 1's stage is free; tile i + 2's rows are placed
    load(i + 2);
    ask();             // tile i + 3
    if (fresh) {
      fresh = false;
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
    }
    const uint32_t kt = smem + (i % kStages) * kStageBytes, vt = kt + kTile * 256;
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
    // ---- masks, running maximum
    const uint64_t mask = (static_cast<uint64_t>(s_mask[(i & 3) * 2 + 1]) << 32) | s_mask[(i & 3) * 2];
    const int pos0 = cur.tile * kTile;
    float mx[2] = {m2[0], m2[1]};
#pragma unroll
    for (int n = 0; n < kNT; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int tk = tok0 + n * 8 + t4 * 2 + (e & 1);
        const bool seen = ((mask >> tk) & 1) && pos0 + tk < lim[e >> 1];
        s[n][e] = seen ? s[n][e] * sl2 : -INFINITY;
        mx[e >> 1] = fmaxf(mx[e >> 1], s[n][e]);
      }
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
    // ---- values.  A new token's value row that an earlier new token must not see would still meet its zero weight
    // in the product, where NaN and infinities survive: such rows (they are looked for among the last T - 1 tokens
    // only) take the second form, one new token at a time, with the rows behind it zeroed.
    bool poisoned = false;
    if (p.T > 1 && pos0 + kTile > cur.len - p.T + 1) {
      bool bad = false;
      for (int x = tid; x < kTile * 16; x += kThreads) {
        const int r = x >> 4;
        if (pos0 + r > cur.len - p.T && pos0 + r < cur.len) {
          const uint4 w = *reinterpret_cast<const uint4 *>(sm + (vt - smem) + row_chunk(r, x & 15));
          const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
          for (int e = 0; e < 4; ++e)
            bad |= (ws[e] & 0x7F80u) == 0x7F80u || (ws[e] & 0x7F800000u) == 0x7F800000u;
        }
      }
      poisoned = __syncthreads_or(bad);
    }
    if (!poisoned) {
#pragma unroll
      for (int k = 0; k < kNT / 2; ++k)
#pragma unroll
        for (int n = 0; n < 16; n += 2) {
          uint32_t b[4];   // tokens k*16 .. +15, channels n*8 .. +15
          ldsm4_t(b, vt + row_chunk(tok0 + k * 16 + (lane & 15), n + (lane >> 4)));
          mma_16816(o[n], pf[k], b[0], b[1]);
          mma_16816(o[n + 1], pf[k], b[2], b[3]);
        }
    } else {
      for (int t = p.T - 1; t >= 0; --t) {
        const int n_t = min(max(cur.len - p.T + t + 1, 0), cur.len);
        for (int x = tid; x < kTile * 16; x += kThreads)
          if (pos0 + (x >> 4) >= n_t)
            *reinterpret_cast<uint4 *>(sm + (vt - smem) + row_chunk(x >> 4, x & 15)) = make_uint4(0u, 0u, 0u, 0u);
        __syncthreads();
        const int row0 = (cur.hr % p.row_blocks) * kRows + 16 * wr + g;
        const bool on0 = row0 / p.G == t, on1 = (row0 + 8) / p.G == t;
#pragma unroll
        for (int k = 0; k < kNT / 2; ++k)
#pragma unroll
          for (int n = 0; n < 16; n += 2) {
            uint32_t b[4];
            ldsm4_t(b, vt + row_chunk(tok0 + k * 16 + (lane & 15), n + (lane >> 4)));
            float x[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
            mma_16816(x[0], pf[k], b[0], b[1]);
            mma_16816(x[1], pf[k], b[2], b[3]);
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              if (on0) { o[n + y][0] += x[y][0]; o[n + y][1] += x[y][1]; }
              if (on1) { o[n + y][2] += x[y][2]; o[n + y][3] += x[y][3]; }
            }
          }
        __syncthreads();
      }
    }
    place();   // tile i + 3's rows, by the page ids asked for before the products

    // ---- the item's (or the stretch's) end: join the warps of each row group, write the rows or the part
    const bool item_ends = cur.tile + 1 == cur.ntiles;
    if (item_ends || i + 1 == ntiles_here) {
      const bool whole = item_ends && cur.tile - i <= 0;   // the item began in this stretch, too
      float l0 = l2[0], l1 = l2[1];
      l0 += __shfl_xor_sync(0xffffffffu, l0, 1);
      l0 += __shfl_xor_sync(0xffffffffu, l0, 2);
      l1 += __shfl_xor_sync(0xffffffffu, l1, 1);
      l1 += __shfl_xor_sync(0xffffffffu, l1, 2);
      __syncthreads();   // tile i has been read: its stage takes the sums
      float *so = reinterpret_cast<float *>(sm + (i % kStages) * kStageBytes);
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
      __syncthreads();
      const int rb = cur.hr % p.row_blocks, h = cur.hr / p.row_blocks;
      const int slot = 2 * blockIdx.x + (cur.tile - i <= 0 ? 1 : 0);
      for (int r = warp; r < kRows; r += 4) {
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
        if (whole) {
          paged_store_row(p, cur.b, t, h * p.G + row % p.G, lane, acc, mm, ll);
        } else {
          float *part = p.parts + (static_cast<size_t>(slot) * kRows + r) * kPagedPartFloats;
          *reinterpret_cast<float4 *>(part + lane * 4) = acc;
          if (lane == 0) *reinterpret_cast<float2 *>(part + kD) = make_float2(mm, ll);
        }
      }
      fresh = true;
    }
    advance(p, cur, ipr);
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
}

// Joins the parts of the items that the stretches cut: CTA (cut i, group of 4 rows), a warp per row.
__global__ void __launch_bounds__(kThreads) paged_join_kernel(PagedArgs p, int rows_per_item) {
  sm100::grid_dependency_wait();
  const int cut = blockIdx.x;
  const int4 j = p.joins[cut];
  const int r = blockIdx.y * 4 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (j.x == 0) return;
  const int rb = j.z % p.row_blocks, h = j.z / p.row_blocks;
  const int row = rb * rows_per_item + r, t = row / p.G;
  if (t >= p.T) return;
  // part 0: the stretch before the cut, in its last slot; part n: the n-th stretch from the cut on, in its first
  auto part = [&](int n) {
    const int slot = n == 0 ? 2 * (cut - 1) + 1 : 2 * (cut + n - 1);
    return p.parts + (static_cast<size_t>(slot) * rows_per_item + r) * kPagedPartFloats;
  };
  float mm = -INFINITY;
  for (int n = lane; n < j.x; n += 32) mm = fmaxf(mm, part(n)[kD]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) mm = fmaxf(mm, __shfl_xor_sync(0xffffffffu, mm, o));
  const float bs = mm == -INFINITY ? 0.f : mm;
  float ll = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int n = 0; n < j.x; ++n) {
    const float *q = part(n);
    const float2 ml = *reinterpret_cast<const float2 *>(q + kD);
    const float4 x = *reinterpret_cast<const float4 *>(q + lane * 4);
    const float c = fast_exp2(ml.x - bs);
    ll += c * ml.y;
    acc.x += c * x.x; acc.y += c * x.y; acc.z += c * x.z; acc.w += c * x.w;
  }
  paged_store_row(p, j.y, t, h * p.G + row % p.G, lane, acc, mm, ll);
}

template <int WR>
cudaError_t launch_paged(PagedArgs a, cudaStream_t stream) {
  static std::mutex mu;
  static uint64_t done = 0;
  if (const cudaError_t e = set_attributes_once(mu, done, [] {
        return cudaFuncSetAttribute(paged_attention_kernel<WR>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
      }))
    return e;
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    sms = 152;
  a.row_blocks = (a.T * a.G + 16 * WR - 1) / (16 * WR);
  const int64_t items = static_cast<int64_t>(a.B) * a.Hk * a.row_blocks;
  const int64_t most = items * std::max<int64_t>(1, (a.max_len + kTile - 1) / kTile);   // tiles there can be
  if (most == items) a.joins = nullptr;   // one tile an item: nothing is cut
  const unsigned grid = static_cast<unsigned>(std::min<int64_t>(most, std::min(2 * sms, kPagedMaxCtas)));
  paged_attention_kernel<WR><<<grid, kThreads, kSmemBytes, stream>>>(a);
  if (const cudaError_t e = cudaGetLastError()) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid, 4 * WR);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return a.joins ? cudaLaunchKernelEx(&cfg, paged_join_kernel, a, 16 * WR) : cudaSuccess;
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
