// Chunked prefill of the gated delta rule on sm_103a.
//
// With chunks of C = 64 tokens, b_t the cumulative log-decay inside a chunk, k^, q^ the l2-normalised keys and
// queries and S the state entering the chunk, the recurrence S_t = (I - beta k^ k^T) e^lambda S_{t-1} + beta k^ v^T is
//
//   A_ri = beta_r k^_r.k^_i e^(b_r - b_i)  (i < r),     L = (I + A)^-1
//   P_ri = q^_r.k^_i e^(b_r - b_i)         (i <= r)
//   R_i  = beta_i (v_i - e^(b_i) S^T k^_i),   U = L R
//   o_r  = scale (e^(b_r) S^T q^_r + (P U)_r),   S' = e^(b_63) S + sum_i e^(b_63 - b_i) k^_i U_i^T
//
// The decay is one number per token, so every product runs on the caller's own bf16 keys and queries and the norms
// and decays are fp32 factors of rows and columns: nothing is rounded that the caller did not round.
//
// Two kernels.  The intra-chunk kernel forms L = (I + A)^-1 and P of every (chunk, value head) at once: 25 KB a block
// instead of the keys', queries' and values' products with L.  The state pass walks a sequence's chunks with S in
// fp32 registers, three products a chunk.
//
// Operands that are not the caller's data are pairs.  S is two bf16 (its rounding, at most 2^-17, is contracted by the chunk).
// L, R and U are two fp16, 22 bits: |L| <= 1, since (I - beta k^ k^T) contracts, and |P| <= 1; R and U carry a power
// of two per value channel that keeps them in fp16's range whatever the values are (from |v| and a bound on the
// channel's state, |S_t|^2 <= |S_(t-1)|^2 + v_t^2); the keys they meet are the caller's, times a power of two per token
// (exact down to 2^-17 of a key's norm).  Final states agree with the 64-bit recurrence to a few 1e-7 (1 to 2e-6 where decays
// are so weak that S's rounding counts), like an fp32 evaluation, where pairs of bf16 throughout leave 3 to 6e-6 and single
// bf16 operands a few 1e-3.  What only an output sees
// is rounded once (P and its U to fp16, S to bf16).
#include <cuda.h>

#include <cuda_fp16.h>

#include <algorithm>
#include <numeric>

#include "kda_hybrid.cuh"

namespace kda {
namespace {

using namespace sm100;

constexpr int kC = 64;
// a block: [L hi ; P ; L lo] (192 rows x 64 tokens, fp16, 128-byte row swizzle) | factors
constexpr uint32_t kBlkP = 8192, kBlkL2 = 16384, kBlkVec = 24576;
constexpr uint32_t kGdnBlkBytes = 26112;
// factors (fp32): beta_i | -beta_i e^(b_i) |k_i|^-1 | scale e^(b_r) |q_r|^-1 | 2^-x_i | 2^(x_i) e^(b_63 - b_i) |k_i|^-1 |
// e^(b_63), with 2^(x_i) the raw key's norm or up to twice that | which rows are taken times kRowScale (k, q: 64 bits each)
constexpr int kVecB = 0, kVecK = 64, kVecQ = 128, kVecX = 192, kVecS = 256, kVecGamma = 320, kVecLong = 324;
static_assert(kBlkVec + 4 * (kVecLong + 4) <= kGdnBlkBytes && (kBlkVec + 4 * kVecLong) % 16 == 0, "block map");
// Keys and queries meet as they are, and products of rows with squares below kRowMost stay inside fp32.  Longer rows (finite
// in bf16 all the same) are taken times a power of two, exactly, wherever they are loaded: their norm takes it back.
constexpr float kRowMost = 1e38f, kRowScale = 8.271806125530277e-25f /* 2^-80 */;
constexpr int kGdnMaxSeqs = 1024;   // sequences per launch (longer batches are split on the host)

// A state pass is serial in a sequence's chunks, so few long sequences leave most of the GPU idle.  They are cut into
// segments of seg chunks.  Within a segment the state is affine in the state S that enters it, S_end = F S + B, and F and
// B are states of the same pass: F is what becomes of the identity without values, B of a zero state with them.  One
// grid runs first segments (as usual: their state is known) and F and B of the inner ones, a small kernel forms
// S_(j+1) = F_j S_j + B_j in fp32, and a second grid runs the segments behind the first from those states.  Where it
// pays, F and B are also kept half way: the second grid then runs inner segments as halves, from S_j and the half-way
// state that the same kernel forms from it, and the last segment is about half as long.
constexpr int kGdnMaxJobs = 256, kGdnMaxSegs = 16;   // jobs per grid, segments per sequence
constexpr int kGdnMaxMats = 400;                     // matrices times heads (64 KB each)
// Chunks of the shortest segment, and what costs in chunks' time: cutting (two more grids, their states), half-way states
// (another grid), a CTA behind another on an SM.  Measured, whole against cut, 16 heads: one sequence of 768 tokens 41 and
// 41 us, of 896 46 and 43, of 1024 51 and 44, 2048 95 and 61, 16384 686 and 285; two of 1024 54 and 57, of 1280 67 and 75 (two
// CTAs per SM), of 1536 78 and 73, of 2048 101 and 90.  Without half-way states and with them: 4096 tokens 98 and 102 us,
// 6000 132 and 134, 8192 170 and 165, 13000 246 and 235, 16384 285 and 266.
constexpr int kSegmentMin = 4, kSegmentExtra = 5, kHalvesExtra = 6, kWaveExtra = 3;
// A piece of a sequence's state pass.  Matrices are numbered per launch; those of a sequence with k inner segments are S_1 ..
// S_(k+1), F_1 .. F_k, and half way B (then the state) and F of each.
struct GdnJob {
  uint16_t seq;
  int16_t src;         // entering state: a matrix, or one of the below
  int16_t dst;         // end: a matrix, or one of the below
  int16_t mid;         // half way, before chunk mid_chunk: a matrix, or none
  int32_t chunk0, chunks, mid_chunk;
};
enum { kFromCaller = -1, kFromZero = -2, kFromIdentity = -3, kToCaller = -1, kToNothing = -2 };

struct GdnPrefillParams {
  CUtensorMap tq, tk, tv, tout; // [tokens, H, 128] bf16, box 64 channels x 1 head x 64 tokens, 128-byte swizzle
  const uint16_t *a, *beta;
  int64_t a_stride, beta_stride;
  const float *A_log, *dt_bias;
  float scale;
  int Hk, Hv, group;
  uint8_t *blocks;              // block (slot g, value head h) at blocks + (g Hv + h) kGdnBlkBytes
  const int32_t *slot_ids;      // indexed by the sequence of the launch
  int num_slots;
  const float *state_in;
  float *state_out_pool, *state_out_dense;
  uint16_t *out;
  int64_t out_stride;
  uint32_t *status;
  int num_seqs;
  int32_t cu[kGdnMaxSeqs + 1];  // first token of each sequence of the launch, and the end of the last
  uint16_t order[kGdnMaxSeqs];  // sequences, longest first
  // segments
  int behind;                   // the entering states come from the grid before
  float *mats;                  // matrix m of head h at mats + (m Hv + h) 128 128
  GdnJob job[kGdnMaxJobs];
};
static_assert(sizeof(GdnPrefillParams) <= 32764, "kernel parameters are limited to 32764 bytes");

// Chunk slots: sequence n's chunks start at slot cu[n] / 64 + n (relative to the launch's first token), which leaves
// each sequence its ceil(len / 64) slots whatever the lengths are.
__host__ __device__ __forceinline__ int first_slot(const GdnPrefillParams &p, int n) { return (p.cu[n] - p.cu[0]) / kC + n; }

__device__ __forceinline__ float2 sub2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 ra, rb, rd;\n\tmov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %5};\n\t"
      "sub.rn.f32x2 rd, ra, rb;\n\tmov.b64 {%0, %1}, rd;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 ra, rb, rd;\n\tmov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %5};\n\t"
      "add.rn.f32x2 rd, ra, rb;\n\tmov.b64 {%0, %1}, rd;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ uint32_t pack_f16x2(float2 x) {
  const __half2 h = __floats2half2_rn(x.x, x.y);
  return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ float2 unpack_f16x2(uint32_t w) { return __half22float2(*reinterpret_cast<const __half2 *>(&w)); }
// Two values as sums of two fp16 each, to 2^-22 (and 2^-25 absolutely).
__device__ __forceinline__ void split2h(float2 x, uint32_t &p1, uint32_t &p2) {
  p1 = pack_f16x2(x);
  p2 = pack_f16x2(sub2(x, unpack_f16x2(p1)));
}
// Two values as sums of two bf16 each, to 2^-18.
__device__ __forceinline__ void split2(float2 x, uint32_t &p1, uint32_t &p2) {
  p1 = pack_bf16x2(x.x, x.y);
  const float2 r = sub2(x, unpack_bf16x2(p1));
  p2 = pack_bf16x2(r.x, r.y);
}

// 16 bytes of a row, times kRowScale
__device__ __forceinline__ void scale_piece(uint8_t *at) {
  uint4 w = *reinterpret_cast<const uint4 *>(at);
  const float2 f = make_float2(kRowScale, kRowScale);
  w.x = pack2(mul2(unpack_bf16x2(w.x), f));
  w.y = pack2(mul2(unpack_bf16x2(w.y), f));
  w.z = pack2(mul2(unpack_bf16x2(w.z), f));
  w.w = pack2(mul2(unpack_bf16x2(w.w), f));
  *reinterpret_cast<uint4 *>(at) = w;
}

// ================================================================ intra-chunk kernel
namespace in {
constexpr int kThreads = 256;   // 8 warps; four CTAs per SM
constexpr int kStride = 68;
constexpr uint32_t OFF_KQ = 0;           // [k ; q], 128 rows x 128 channels: consumed by the first product; then
constexpr uint32_t OFF_A = 0;            // A fp32 [64][68], turned into (I + A)^-1 in place
constexpr uint32_t OFF_BLK = 17408;      // the block's image
constexpr uint32_t OFF_SMALL = OFF_BLK + kGdnBlkBytes;
constexpr uint32_t SM_NORM = 0 /* [128]: 1 / |k_r|, 1 / |q_r| */, SM_BETA = 512, SM_BI = 768, SM_BF = 1024 /* b, whole and
                   fractional part */, SM_UP = 1280 /* 2^-b */, SM_POW = 1536 /* 2^-x */, SM_BAR = 1792, SM_TMEM = 1808, SM_ABORT = 1812,
                   SM_LONG = 1824 /* a bit a row of [k ; q]: its squares pass kRowMost */, SM_END = 1840;
constexpr uint32_t kSmemBytes = OFF_SMALL + SM_END + 1024;
static_assert(OFF_BLK == 64 * kStride * 4 && OFF_BLK % 1024 == 0 && OFF_SMALL >= 32768, "shared memory map");
static_assert(SM_POW + 256 <= SM_BAR && SM_BAR + 2 * 8 <= SM_TMEM && SM_TMEM + 4 <= SM_ABORT && SM_ABORT + 4 <= SM_LONG &&
                  SM_LONG + 16 <= SM_END,
              "small part of the shared memory map");
static_assert(4 * (kSmemBytes + 1024) <= 233472, "four CTAs per SM");
constexpr uint32_t kTmemCols = 128;
// Decays of a chunk down to 2^-kFactorRange are split into a row's and a column's factor (2^b_r and 2^-b_i stay far
// inside fp32); beyond that each entry takes its own exponential.
constexpr float kFactorRange = 60.f;
}  // namespace in

// 16 x 8 tile of X Y for X (16 x 8 KS), Y (8 KS x 8), fp32 with row stride in::kStride, on TF32 tensor cores.  Each operand
// is a pair of TF32 (the hardware drops the bits below a TF32's): x1 y1 + x1 y2 + x2 y1 leaves about 2^-21.
template <int KS>
__device__ __forceinline__ void mm_tile(float (&d)[4], const float *X, const float *Y, int lane) {
  const int g = lane >> 2, t = lane & 3;
  float c[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int k = 0; k < KS; ++k) {
    const float *xa = X + g * in::kStride + 8 * k + t;
    const float *yb = Y + (8 * k + t) * in::kStride + g;
    const float x[4] = {xa[0], xa[8 * in::kStride], xa[4], xa[8 * in::kStride + 4]};
    const float y[2] = {yb[0], yb[4 * in::kStride]};
    uint32_t xh[4], yh[2], xl[4], yl[2];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      xh[i] = __float_as_uint(x[i]) & 0xFFFFE000u;
      xl[i] = __float_as_uint(x[i] - __uint_as_float(xh[i]));
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      yh[i] = __float_as_uint(y[i]) & 0xFFFFE000u;
      yl[i] = __float_as_uint(y[i] - __uint_as_float(yh[i]));
    }
    mma_1688_tf32(d, xh[0], xh[1], xh[2], xh[3], yh[0], yh[1]);
    mma_1688_tf32(c, xh[0], xh[1], xh[2], xh[3], yl[0], yl[1]);
    mma_1688_tf32(c, xl[0], xl[1], xl[2], xl[3], yh[0], yh[1]);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) d[i] += c[i];
}
__device__ __forceinline__ void st_tile(float *D, const float (&d)[4], float sgn, int lane) {
  const int g = lane >> 2, t = lane & 3;
  *reinterpret_cast<float2 *>(D + g * in::kStride + 2 * t) = make_float2(sgn * d[0], sgn * d[1]);
  *reinterpret_cast<float2 *>(D + (g + 8) * in::kStride + 2 * t) = make_float2(sgn * d[2], sgn * d[3]);
}
// the same tile, times sgn, into the two parts of L (rows row0.., columns col0..)
__device__ __forceinline__ void st_tile_l(uint8_t *blk, int row0, int col0, const float (&d)[4], float sgn, int lane) {
  const int g = lane >> 2, c = col0 + 2 * (lane & 3);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    uint32_t p1, p2;
    split2h(make_float2(sgn * d[2 * i], sgn * d[2 * i + 1]), p1, p2);
    uint8_t *at = blk + swz_offset(64, row0 + g + 8 * i, c);
    *reinterpret_cast<uint32_t *>(at) = p1;
    *reinterpret_cast<uint32_t *>(at + kBlkL2) = p2;
  }
}
// One CTA per (chunk slot, key head): the products of the chunk's keys and queries serve every value head of the group.
// Short dependent phases on one chunk, hidden by four CTAs per SM (TMEM and shared memory hold no fifth); its traffic is
// the keys and queries in and 25 KB a value head out.  Measured: 2048 x 8 tokens, 16 heads 59 us (issue slots 50 % busy,
// 3.3 TB/s).  Neither issue nor memory is full: what binds has not been measured phase by phase (phases in which two or
// four of the eight warps work, seven barriers a value head).  Phases in parallel warps with two barriers fewer took 61 us.
__global__ void __launch_bounds__(in::kThreads, 4) gdn_intra_kernel(const __grid_constant__ GdnPrefillParams prm) {
  using namespace in;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *sm = smem_raw + (-smem_u32(smem_raw) & 1023u);   // (an offset, so that accesses stay shared-memory ones)
  uint8_t *small = sm + OFF_SMALL;
  float *s_norm = reinterpret_cast<float *>(small + SM_NORM);
  float *s_beta = reinterpret_cast<float *>(small + SM_BETA);
  float *s_bi = reinterpret_cast<float *>(small + SM_BI);
  float *s_bf = reinterpret_cast<float *>(small + SM_BF);
  float *s_up = reinterpret_cast<float *>(small + SM_UP);
  float *s_pow = reinterpret_cast<float *>(small + SM_POW);
  uint64_t *bar_in = reinterpret_cast<uint64_t *>(small + SM_BAR);
  uint64_t *bar_mma = bar_in + 1;
  uint32_t *s_tmem = reinterpret_cast<uint32_t *>(small + SM_TMEM);
  volatile uint32_t *s_abort = reinterpret_cast<volatile uint32_t *>(small + SM_ABORT);
  uint32_t *s_long = reinterpret_cast<uint32_t *>(small + SM_LONG);
  uint8_t *s_blk = sm + OFF_BLK;
  float *sA = reinterpret_cast<float *>(sm + OFF_A);

  // (TMEM is taken behind the wait: a grid before this one may still be taking its own)
  grid_dependency_wait();
  grid_launch_dependents();   // the state pass may take SMs as this grid leaves them, and read the caller's tensors
  const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);   // (uniform in the warp)
  const int hk = blockIdx.x % prm.Hk, slot = blockIdx.x / prm.Hk;
  int n = 0;   // the slot's sequence: the last that starts at or before it
  for (int hi = prm.num_seqs - 1; n < hi;) {
    const int mid = (n + hi + 1) >> 1;
    if (first_slot(prm, mid) <= slot) n = mid; else hi = mid - 1;
  }
  const int tok0 = prm.cu[n] + (slot - first_slot(prm, n)) * kC;
  const int valid = min(kC, prm.cu[n + 1] - tok0);
  if (valid <= 0) return;   // a slot between two sequences

  const auto fetch = [&] {
    mbar_arrive_expect_tx(bar_in, 32768);
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      tma_load_3d(sm + OFF_KQ + 16384 * x, &prm.tk, 64 * x, hk, tok0, bar_in);
      tma_load_3d(sm + OFF_KQ + 16384 * x + 8192, &prm.tq, 64 * x, hk, tok0, bar_in);
    }
  };
  if (tid == 0) {
    mbar_init(bar_in, 1);
    mbar_init(bar_mma, 1);
    *s_abort = 0;
    fence_mbar_init();
    fetch();
  }
  if (warp == 1) {
    tmem_alloc(s_tmem, kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *s_tmem;

  // ---- [k ; q] [k ; q]^T: rows 0..63 k.k, rows 64..127 q.k; its diagonal holds the squared norms
  const auto multiply = [&] {
    const uint64_t kq = desc_kmajor_base(smem_u32(sm + OFF_KQ));
    const uint32_t id = idesc_bf16(128, 128, false, false);
#pragma unroll
    for (int s = 0; s < 8; ++s) mma_bf16(tmem, kq + kmajor_step(128, s), kq + kmajor_step(128, s), id, s > 0);
    mma_commit(bar_mma);
  };
  if (tid == 0) {
    wait_or_abort(bar_in, 0, s_abort, prm.status);
    multiply();
  }
  __syncwarp();
  const int q4 = warp & 3, ib = warp >> 2;   // TMEM lane quadrant, half of the 64 key columns
  const uint32_t lanes = tmem + (static_cast<uint32_t>(q4 * 32) << 16);

  // ---- the rows' norms (again: once long rows have been scaled), and what stays zero in the blocks
  const auto norms = [&](bool again) {
    wait_or_abort(bar_mma, again, s_abort, prm.status);
    tc_fence_after();
    if (warp < 4) {   // row 32 q4 + lane: its diagonal entry
      uint32_t v[32];
      tmem_ld16_async(lanes + 32 * q4, v);
      tmem_ld16_async(lanes + 32 * q4 + 16, v + 16);
      tmem_wait_ld();
      tmem_tie<32>(v);
#pragma unroll
      for (int half = 16; half > 0; half >>= 1) {   // entry `lane`: a bit of it at a time
        const bool up = lane & half;
#pragma unroll
        for (int e = 0; e < half; ++e) v[e] = up ? v[e + half] : v[e];
      }
      const float d = __uint_as_float(v[0]);
      const int r = 32 * q4 + lane;
      const bool in = (r & 63) < valid;
      // (a row that has been scaled leaves the 1e-6 far below its squares)
      s_norm[r] = in ? rsqrtf(again && s_long[q4] >> lane & 1 ? d : d + kL2Eps) : 0.f;
      // a power of two that brings the raw key's norm to (1/2, 1] (a zero key: any)
      if (r < 64) s_pow[r] = in ? __uint_as_float(__float_as_uint(rsqrtf(fmaxf(d, 1e-36f))) & 0x7F800000u) : 1.f;
      if (!again) {
        const uint32_t mine = __ballot_sync(0xffffffffu, in && !(d <= kRowMost));
        if (lane == 0) s_long[q4] = mine;
      }
    } else {
      // zeros above the diagonal of L's parts and of P (the value heads of the group leave them): 6 blocks x 16
      // rows x two 16-byte pieces of each
      for (int x = tid - 128; x < 3 * 192; x += 128) {
        const int which = x / 192, y = x % 192, b6 = y >> 5, rr = (y >> 1) & 15, hc = y & 1;
        const int I = b6 < 3 ? 0 : b6 < 5 ? 1 : 2;
        const int J = b6 < 3 ? b6 + 1 : b6 < 5 ? b6 - 1 : 3;
        *reinterpret_cast<uint4 *>(s_blk + 8192 * which + swz_offset(64, 16 * I + rr, 16 * J + 8 * hc)) = make_uint4(0, 0, 0, 0);
      }
    }
  };

  for (int gh = 0; gh < prm.group; ++gh) {
    const int h = hk * prm.group + gh;
    // ---- warp 7: log2 of the decays, summed exactly in fixed point (32 fractional bits); beta
    // A decay below 2^-160 is 0 in fp32 alone and in any product; the bound keeps the sums small.
    if (warp == 7) {
      const float rate = expf(prm.A_log[h]) * kLog2e, bias = prm.dt_bias[h];
      int64_t b[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = 2 * lane + e;
        float lam = 0.f, be = 0.f;
        if (r < valid) {
          const int64_t t = tok0 + r;
          lam = -rate * softplus(bf16_bits_to_f32(prm.a[t * prm.a_stride + h]) + bias);
          be = 1.0f / (1.0f + expf(-bf16_bits_to_f32(prm.beta[t * prm.beta_stride + h])));
          if (lam != lam) be = lam;   // a decay that is no number reaches everything behind it through beta
          lam = lam < -160.f ? -160.f : lam;
        }
        const float whole = rintf(lam);
        b[e] = lam == lam ? static_cast<int64_t>(static_cast<int>(whole)) * 4294967296ll +
                                static_cast<int64_t>((lam - whole) * 4294967296.0f)
                          : 0;
        s_beta[r] = be;
      }
      int64_t sum = b[0] + b[1];
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t u = __shfl_up_sync(0xffffffffu, sum, o);
        if (lane >= o) sum += u;
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int64_t x = e ? sum : sum - b[1];
        const float bi = static_cast<float>(static_cast<int>(x >> 32));
        const float bf = static_cast<float>(static_cast<uint32_t>(x)) * 2.3283064365386963e-10f;
        s_bi[2 * lane + e] = bi;
        s_bf[2 * lane + e] = bf;
        s_up[2 * lane + e] = fast_exp2(-bi) * fast_exp2(-bf);   // (their sum would lose bits of bf)
      }
    }
    if (gh == 0) norms(false);
    __syncthreads();
    if (gh == 0) {
      const uint4 rows4 = *reinterpret_cast<const uint4 *>(s_long);
      if (rows4.x | rows4.y | rows4.z | rows4.w) {   // the tiles once more (the zeros are over them), long rows scaled
        fence_async_smem();
        tc_fence_before();
        __syncthreads();
        if (tid == 0) fetch();
        __syncwarp();
        wait_or_abort(bar_in, 1, s_abort, prm.status);
        const int r = tid >> 1;
        if (s_long[r >> 5] >> (r & 31) & 1)
          for (int c = 0; c < 64; c += 8) scale_piece(sm + OFF_KQ + swz_offset(128, r, 64 * (tid & 1) + c));
        fence_async_smem();
        __syncthreads();
        if (tid == 0) {
          tc_fence_after();
          multiply();
        }
        __syncwarp();
        norms(true);
        __syncthreads();
      }
    }

    // ---- A (fp32) and P (fp16) from TMEM; the block's factors
    {
      const bool is_p = q4 >= 2;
      const int r = (q4 & 1) * 32 + lane;
      const float bi = s_bi[r], bf = s_bf[r];
      const float rowf = is_p ? s_norm[64 + r] : s_beta[r] * s_norm[r];
      const bool factors = s_bi[63] > -kFactorRange;   // (b falls along the chunk)
      const float down = rowf * (fast_exp2(bi) * fast_exp2(bf));
      if ((q4 & 1) >= ib) {   // (rows 0..31, columns 32..63 lie above the diagonal)
        const int lim = r < valid ? r - 32 * ib + (is_p ? 1 : 0) : 0;   // kept: i < r (A), i <= r (P)
        const bool masked = __any_sync(0xffffffffu, lim < 32);   // (not below the diagonal in a full chunk)
        uint32_t v[32];
        tmem_ld16_async(lanes + 32 * ib, v);
        tmem_ld16_async(lanes + 32 * ib + 16, v + 16);
        tmem_wait_ld();
        tmem_tie<32>(v);
#pragma unroll
        for (int e0 = 0; e0 < 32; e0 += 8) {
          float x[8];
#pragma unroll
          for (int e = 0; e < 8; e += 4) {
            const int i = 32 * ib + e0 + e;
            const float4 nk = *reinterpret_cast<const float4 *>(s_norm + i);
            const float n4[4] = {nk.x, nk.y, nk.z, nk.w};
            if (factors) {
              const float4 up = *reinterpret_cast<const float4 *>(s_up + i);
              const float u4[4] = {up.x, up.y, up.z, up.w};
#pragma unroll
              for (int z = 0; z < 4; ++z) x[e + z] = (__uint_as_float(v[e0 + e + z]) * down) * (n4[z] * u4[z]);
            } else {
#pragma unroll
              for (int z = 0; z < 4; ++z)
                x[e + z] = __uint_as_float(v[e0 + e + z]) * (rowf * n4[z]) * fast_exp2((bi - s_bi[i + z]) + (bf - s_bf[i + z]));
            }
          }
          if (masked) {
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] = e0 + e < lim ? x[e] : 0.f;
          }
          if (is_p) {
            *reinterpret_cast<uint4 *>(s_blk + kBlkP + swz_offset(64, r, 32 * ib + e0)) =
                make_uint4(pack_f16x2(make_float2(x[0], x[1])), pack_f16x2(make_float2(x[2], x[3])),
                           pack_f16x2(make_float2(x[4], x[5])), pack_f16x2(make_float2(x[6], x[7])));
          } else {
            float *dst = sA + r * kStride + 32 * ib + e0;
            *reinterpret_cast<float4 *>(dst) = make_float4(x[0], x[1], x[2], x[3]);
            *reinterpret_cast<float4 *>(dst + 4) = make_float4(x[4], x[5], x[6], x[7]);
          }
        }
      } else {   // one of the two warps without entries: the block's factors, two rows a lane
        if (!is_p) {
          float *vec = reinterpret_cast<float *>(s_blk + kBlkVec);
#pragma unroll
          for (int e = 0; e < 64; e += 32) {
            const int t = lane + e;
            const float eb = fast_exp2(s_bi[t]) * fast_exp2(s_bf[t]);
            vec[kVecB + t] = s_beta[t];
            vec[kVecK + t] = -s_beta[t] * s_norm[t] * eb;
            vec[kVecQ + t] = prm.scale * s_norm[64 + t] * eb;
            vec[kVecX + t] = s_pow[t];
            vec[kVecS + t] = s_norm[t] / s_pow[t] * fast_exp2((s_bi[63] - s_bi[t]) + (s_bf[63] - s_bf[t]));
            if (t == 63) vec[kVecGamma] = eb;
            if (t < 4) reinterpret_cast<uint32_t *>(vec)[kVecLong + t] = s_long[t];
          }
        }
      }
    }
    __syncthreads();

    // ---- L = (I + A)^-1: 16 x 16 diagonal inverses D_R by substitution, then
    //   L^-1_10 = -D_1 A_10 D_0,  L^-1_32 = -D_3 A_32 D_2,  L^-1 (rows 32.., cols ..31) = -I_2 A_(23,01) I_1
    // in place in the A tile, temporaries in its unused upper part; every block goes to L's parts as it is made.
    if (tid < 64) {   // thread = (block R, column jc)
      const int R = tid >> 4, jc = tid & 15;
      float *a = sA + (16 * R) * kStride + 16 * R;
      float xs[16];
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        float4 row[4];
#pragma unroll
        for (int m = 0; m < r; m += 4) row[m / 4] = *reinterpret_cast<const float4 *>(a + r * kStride + m);
        float acc[4] = {r == jc ? 1.f : 0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int m = 0; m < r; ++m) {
          const float am = m % 4 == 0 ? row[m / 4].x : m % 4 == 1 ? row[m / 4].y : m % 4 == 2 ? row[m / 4].z : row[m / 4].w;
          acc[m & 3] = fmaf(-am, xs[m], acc[m & 3]);
        }
        xs[r] = (acc[0] + acc[1]) + (acc[2] + acc[3]);
      }
      __syncwarp();   // the block's entries of A have been read
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        a[i * kStride + jc] = xs[i];
        const __half hi = __float2half_rn(xs[i]);
        uint8_t *at = s_blk + swz_offset(64, 16 * R + i, 16 * R + jc);
        *reinterpret_cast<__half *>(at) = hi;
        *reinterpret_cast<__half *>(at + kBlkL2) = __float2half_rn(xs[i] - __half2float(hi));
      }
    }
    __syncthreads();
    if (warp < 4) {
      const int lo = warp < 2 ? 0 : 32, nj = warp & 1;
      float d[4] = {0.f, 0.f, 0.f, 0.f};
      mm_tile<2>(d, sA + (lo + 16) * kStride + lo, sA + lo * kStride + lo + 8 * nj, lane);
      st_tile(sA + lo * kStride + lo + 16 + 8 * nj, d, 1.f, lane);
      if (warp < 2) named_bar_sync<5>(64); else named_bar_sync<6>(64);   // A_10 (A_32) has been read
      float e[4] = {0.f, 0.f, 0.f, 0.f};
      mm_tile<2>(e, sA + (lo + 16) * kStride + lo + 16, sA + lo * kStride + lo + 16 + 8 * nj, lane);
      st_tile(sA + (lo + 16) * kStride + lo + 8 * nj, e, -1.f, lane);
      st_tile_l(s_blk, lo + 16, lo + 8 * nj, e, -1.f, lane);
    }
    __syncthreads();
    {   // Z = A_(23,01) I_1 -> rows 0..31, cols 32..63
      const int mi = warp >> 2, nj = warp & 3;
      float d[4] = {0.f, 0.f, 0.f, 0.f};
      if (nj < 2) mm_tile<4>(d, sA + (32 + 16 * mi) * kStride, sA + 8 * nj, lane);
      else mm_tile<2>(d, sA + (32 + 16 * mi) * kStride + 16, sA + 16 * kStride + 8 * nj, lane);
      st_tile(sA + (16 * mi) * kStride + 32 + 8 * nj, d, 1.f, lane);
    }
    __syncthreads();
    {
      const int mi = warp >> 2, nj = warp & 3;
      float d[4] = {0.f, 0.f, 0.f, 0.f};
      if (mi) mm_tile<4>(d, sA + 48 * kStride + 32, sA + 32 + 8 * nj, lane);
      else mm_tile<2>(d, sA + 32 * kStride + 32, sA + 32 + 8 * nj, lane);
      st_tile_l(s_blk, 32 + 16 * mi, 8 * nj, d, -1.f, lane);
    }
    fence_async_smem();
    __syncthreads();
    if (tid == 0) {
      bulk_store(prm.blocks + (static_cast<size_t>(slot) * prm.Hv + h) * kGdnBlkBytes, s_blk, kGdnBlkBytes);
      bulk_commit();
      bulk_wait_read();
    }
    if (gh + 1 < prm.group) __syncthreads();   // the block's image is free for the next value head
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// ================================================================ state pass
// CTA = (sequence, value head).  Products run transposed (TMEM lane = value channel, M = 128), so that the operands a
// chunk makes (S, R, U) go back to TMEM in the lanes they were read from and only the caller's tiles and the block come
// from shared memory (a 16-deep step of N columns takes 32 cycles at N = 64 and 64 at N = 128, but one thread issues one
// in 46: two warps issue, each to accumulators of its own that the epilogue adds):
//   KU = S^T k^T                (S hi by one warp, S lo by the other; N = 64 tokens, K = 128 channels)
//   QS = S^T q^T                (S hi)
//   R^T = beta (v^T - e^b/|k| KU)
//   U = R^T L^T                 (R hi L hi, R hi L lo, R lo L hi; N = 64, K = 64 tokens)
//   OT = U^T P^T                (U hi; N = 64, K = 64),   o = scale e^b/|q| QS + scale OT
//   U'^T = 2^x e^(b_63 - b)/|k| U
//   D = U'^T (2^-x k)           (U' hi, U' lo; N = 128 channels, K = 64),          S = e^(b_63) S + D
//   VT = v^T 1                  (an identity as the other operand: v in the lanes that need it)
// Sixteen epilogue warps (warp w: lanes 32 (w % 4).., quarter w / 4 of the columns; 32 state entries a thread), the two
// issuing warps, one that feeds chunks through two stages, brings the next to L2 and stores the output, and one that goes
// ahead of them all over v for the channels' scales.  The serial path of a chunk is KU -> R -> U -> U' -> D -> S; what it does not need runs
// beside it: VT under S's epilogue, QS under R's, the fp16 keys under U, OT and the output under D.  Bound by that path:
// 2.6 us a chunk on one long sequence, 3.0 with every SM at work (2048 x 8 tokens, 16 heads: 96 us; tensor pipe 35 %, issue 46 %, DRAM
// 48 % busy).  Fetching tokens a chunk earlier, with more scales in flight, took 100 us.
namespace ch {
constexpr int kWorkers = 512, kThreads = kWorkers + 128;
constexpr int kIssuer = 16, kProducer = 18, kScaler = 19;   // warps (two that issue)
constexpr uint32_t ST_V = 32768, ST_BLK = 49152, kStage = 75776;   // [k ; q] | v | block, a multiple of 1024
constexpr uint32_t kStageLoad = ST_BLK + kGdnBlkBytes;
constexpr uint32_t OFF_ONE = 2 * kStage;          // identity, 64 x 64 bf16
constexpr uint32_t OFF_K16 = OFF_ONE + 8192;      // the chunk's keys times 2^-x in fp16 (64 rows x 128 channels)
constexpr uint32_t OFF_OUT = OFF_K16 + 16384;     // output on its way out (64 rows x 128 channels)
constexpr uint32_t OFF_SMALL = OFF_OUT + 16384;
constexpr uint32_t SM_BAR = 0 /* the barriers below */, SM_TMEM = 144, SM_ABORT = 148, SM_SIG = 256 /* [2][128] */, SM_INV = 1280 /* [2][128] */, SM_END = 2304;
// mbarriers: landed in stage 0, 1: all but v, v (which goes first, for the scales); scales of even, odd chunks; products done (first, second, state's, v's, output's); output
// tile free; long rows scaled (both issuing warps) | the workers' warps: S, R, U' in place, stage done with, output in its tile
enum { B_FULL = 0, B_VAL = 2, B_SCALE = 4, B_M1 = 6, B_M2, B_M3, B_V, B_O, B_OUT, B_LONG, B_S, B_R, B_U, B_FREE, B_TILE, kBarriers };
constexpr uint32_t kSmemBytes = OFF_SMALL + SM_END + 1024;
static_assert(kSmemBytes <= 232448 && kStage >= kStageLoad && kStage % 1024 == 0, "shared memory map");
static_assert(SM_BAR + 8 * kBarriers <= SM_TMEM && SM_TMEM + 4 <= SM_ABORT && SM_ABORT + 4 <= SM_SIG &&
                  SM_SIG + 1024 <= SM_INV && SM_INV + 1024 <= SM_END,
              "small part of the shared memory map");
constexpr uint32_t TM_KU = 0 /* two of 64 */, TM_D = 0 /* 128, over KU */, TM_U = 128 /* two of 64 */, TM_OT = 128 /* over U */,
                   TM_V = 192 /* over U */, TM_QS = 256, TM_S = 320 /* two of 64 */, TM_UH = 320 /* 32, over S */,
                   TM_R = 448 /* two of 32 */, kTmemCols = 512;
}  // namespace ch
// A CTA of the state pass takes all of an SM's TMEM, possibly before the intra-chunk grid is done: the two never share one.
static_assert(ch::kSmemBytes + in::kSmemBytes + 2048 > 233472, "no SM holds CTAs of both");

__device__ __forceinline__ void bulk_prefetch(const void *src, uint32_t bytes) {
  asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(reinterpret_cast<uint64_t>(src)), "r"(bytes) : "memory");
}
// one arrival for the warp, once its lanes' writes are done (no branch)
__device__ __forceinline__ void warp_arrive(uint64_t *bar) {
  __syncwarp();
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.eq.u32 p, %1, 0;\n\t"
      "@p mbarrier.arrive.shared::cta.b64 _, [%0];\n\t}"
      ::"r"(smem_u32(bar)), "r"(threadIdx.x & 31)
      : "memory");
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t *v) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};"
               ::"r"(taddr), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}
// 16 lanes x 16 columns of 32 bits in the fragments of a 16 x 8 matrix product: registers 0, 1 and 2, 3 hold rows lane / 4
// and lane / 4 + 8, columns 2 (lane % 4), + 1; registers 4 .. 7 the same of the next 8 columns
__device__ __forceinline__ void tmem_ld_frag(uint32_t taddr, uint32_t *r) {
  asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr));
}
// kind::f16 with fp16 operands
__host__ __device__ constexpr uint32_t idesc_f16(int M, int N, bool a_mn_major, bool b_mn_major) {
  return idesc_bf16(M, N, a_mn_major, b_mn_major) & ~((1u << 7) | (1u << 10));
}

template <bool SEGMENTS>
__global__ void __launch_bounds__(ch::kThreads, 1) gdn_chain_kernel(const __grid_constant__ GdnPrefillParams prm) {
  using namespace ch;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *sm = smem_raw + (-smem_u32(smem_raw) & 1023u);   // (an offset, so that accesses stay shared-memory ones)
  uint8_t *small = sm + OFF_SMALL;
  uint64_t *bar = reinterpret_cast<uint64_t *>(small + SM_BAR);
  uint32_t *s_tmem = reinterpret_cast<uint32_t *>(small + SM_TMEM);
  volatile uint32_t *s_abort = reinterpret_cast<volatile uint32_t *>(small + SM_ABORT);
  float *s_sig = reinterpret_cast<float *>(small + SM_SIG), *s_inv = reinterpret_cast<float *>(small + SM_INV);
  const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);   // (uniform in the warp)

  const int h = blockIdx.x % prm.Hv, hk = h / prm.group;
  GdnJob job = {};
  if (SEGMENTS) job = prm.job[blockIdx.x / prm.Hv];
  const int n = SEGMENTS ? job.seq : prm.order[blockIdx.x / prm.Hv];
  const bool map = SEGMENTS && job.src == kFromIdentity;   // (F: no values)
  int t0 = prm.cu[n], len = prm.cu[n + 1] - t0, chunk0 = 0;
  if (SEGMENTS) {
    chunk0 = job.chunk0;
    t0 += chunk0 * kC;
    len = min(len - chunk0 * kC, job.chunks * kC);
  }
  const int nchunks = (len + kC - 1) / kC;
  // a segment whose entering state is known has outputs; the others' F and B do not
  const bool known = !SEGMENTS || job.src >= kFromCaller;
  int pool_slot = 0;
  if (prm.slot_ids) {
    pool_slot = prm.slot_ids[n];
    if (pool_slot < 0 || pool_slot >= prm.num_slots) {
      if (tid == 0) {
        atomicOr(prm.status, KDA_DEVICE_BAD_SLOT);
        grid_dependency_wait();   // this grid's end implies the intra-chunk grid's on every path
      }
      return;
    }
  }
  const size_t pool_at = (static_cast<size_t>(pool_slot) * prm.Hv + h) * kD * kD;
  const float *src = prm.state_in ? prm.state_in + pool_at : nullptr;
  float *dst = prm.state_out_pool ? prm.state_out_pool + pool_at
                                  : prm.state_out_dense + (static_cast<size_t>(n) * prm.Hv + h) * kD * kD;
  float *mid = nullptr;
  if (SEGMENTS) {
    const auto mat = [&](int m) { return prm.mats + (static_cast<size_t>(m) * prm.Hv + h) * kD * kD; };
    if (job.src != kFromCaller) src = job.src >= 0 ? mat(job.src) : nullptr;
    if (job.dst != kToCaller) dst = job.dst >= 0 ? mat(job.dst) : nullptr;
    if (job.mid >= 0) mid = mat(job.mid);
  }
  if (SEGMENTS && prm.behind) grid_dependency_wait();
  // epilogue thread: value channel d (TMEM lane), key channels 32 cg .. + 31 of the state, tokens 16 cg .. + 15 of a chunk
  const bool worker = warp < kIssuer;
  const int quad = warp & 3, cg = warp >> 2, d = 32 * quad + lane;
  float S[32];
  if (worker) {
#pragma unroll
    for (int e = 0; e < 32; ++e) S[e] = src ? src[(32 * cg + e) * kD + d] : map && 32 * cg + e == d ? 1.f : 0.f;
  }
  if (nchunks > 0) {
    if (tid == 0) {
      for (int i = 0; i < kBarriers; ++i) mbar_init(&bar[i], i >= B_S ? 16 : i == B_M1 || i == B_M2 || i == B_LONG ? 2 : 1);   // (two issuers)
      *s_abort = 0;
      fence_mbar_init();
    }
    if (warp == kProducer) {
      tmem_alloc(s_tmem, kTmemCols);
      tmem_relinquish();
    }
    if (worker && src) {   // the entering state's 1-norms, a quarter of the key channels each
      float sum = 0.f;
#pragma unroll
      for (int e = 0; e < 32; ++e) sum += fabsf(S[e]);
      reinterpret_cast<float *>(sm + OFF_OUT)[128 * cg + d] = sum;
    }
    if (worker) {   // the identity: row tid / 8, the 16 bytes with columns 8 (tid % 8) ..
      const int r = tid >> 3, pc = tid & 7, w = (r & 7) >> 1;
      const uint32_t one = (r >> 3) != pc ? 0u : (r & 1) ? 0x3F800000u : 0x00003F80u;
      *reinterpret_cast<uint4 *>(sm + OFF_ONE + swz_offset(64, r, 8 * pc)) =
          make_uint4(w == 0 ? one : 0u, w == 1 ? one : 0u, w == 2 ? one : 0u, w == 3 ? one : 0u);
      if (map) {   // no values
        for (int i = tid; i < 2048; i += kWorkers)
          *reinterpret_cast<uint4 *>(sm + (i >> 10) * kStage + ST_V + 16 * (i & 1023)) = make_uint4(0, 0, 0, 0);
      }
      fence_async_smem();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *s_tmem;

    if (warp == kProducer) {
      // ------------------------------------------------------------ chunks -> stages, output tiles -> the caller's rows
      const uint8_t *blk = prm.blocks + (static_cast<size_t>(first_slot(prm, n) + chunk0) * prm.Hv + h) * kGdnBlkBytes;
      const size_t step = static_cast<size_t>(prm.Hv) * kGdnBlkBytes;
      auto load = [&](int c) {
        uint8_t *st = sm + (c & 1) * kStage;
        uint64_t *full = &bar[B_FULL + (c & 1)], *val = &bar[B_VAL + (c & 1)];
        const int tok = t0 + c * kC;
        if (map) {
          mbar_arrive(val);
        } else {
          mbar_arrive_expect_tx(val, 16384);
#pragma unroll
          for (int x = 0; x < 2; ++x) tma_load_3d(st + ST_V + 8192 * x, &prm.tv, 64 * x, h, tok, val);
        }
        mbar_arrive_expect_tx(full, kStageLoad - 16384);
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          tma_load_3d(st + 16384 * x, &prm.tk, 64 * x, hk, tok, full);
          tma_load_3d(st + 16384 * x + 8192, &prm.tq, 64 * x, hk, tok, full);
        }
        if (c == 0) grid_dependency_wait();   // the blocks are the intra-chunk grid's
        bulk_load(st + ST_BLK, blk + c * step, kGdnBlkBytes, full);
      };
      if (lane == 0) {
        load(0);
        if (nchunks > 1) load(1);
      }
      __syncwarp();
      for (int c = 0; c < nchunks; ++c) {
        const int valid = min(kC, len - c * kC), tok = t0 + c * kC;
        if (known) wait_or_abort(&bar[B_TILE], c & 1, s_abort, prm.status);   // chunk c's output is in its tile
        if (!known) {
        } else if (valid == kC) {
          if (lane == 0) {
            tma_store_3d(&prm.tout, 0, h, tok, sm + OFF_OUT);
            tma_store_3d(&prm.tout, 64, h, tok, sm + OFF_OUT + 8192);
            bulk_commit();
          }
        } else {   // a ragged last chunk: its own rows alone
          for (int i = lane; i < valid * 16; i += 32) {
            const int r = i >> 4, cc = i & 15;
            *reinterpret_cast<uint4 *>(prm.out + static_cast<int64_t>(tok + r) * prm.out_stride + h * kD + 8 * cc) =
                *reinterpret_cast<const uint4 *>(sm + OFF_OUT + swz_offset(64, r, 8 * cc));
          }
        }
        __syncwarp();
        wait_or_abort(&bar[B_FREE], c & 1, s_abort, prm.status);   // chunk c is done with its stage
        if (lane == 0) {
          if (c + 2 < nchunks && !*s_abort) load(c + 2);
          if (c + 3 < nchunks) {   // the one behind it, into L2
            const int tok3 = tok + 3 * kC;
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              tma_prefetch_3d(&prm.tk, 64 * x, hk, tok3);
              tma_prefetch_3d(&prm.tq, 64 * x, hk, tok3);
              tma_prefetch_3d(&prm.tv, 64 * x, h, tok3);
            }
            bulk_prefetch(blk + (c + 3) * step, kGdnBlkBytes);
          }
          if (known) {
            bulk_wait_read();
            mbar_arrive(&bar[B_OUT]);   // the output tile is free
          }
        }
        __syncwarp();
      }
      if (lane == 0) bulk_wait_all();
      // (every chunk was waited for by the issuing warps; after a timeout the copies in flight are waited for here)
      if (*s_abort) {
        for (int i = 0; i < 4; ++i) {
          mbar_wait(&bar[B_FULL + i], 0);
          mbar_wait(&bar[B_FULL + i], 1);
        }
      }
      __syncwarp();
    } else if (warp == kScaler) {
      // ------------------------------------------------------------ the channels' scales, a chunk ahead
      // |R|, |U| <= |v| + |S| within the chunk < 2^(e + 1) -> below 2^14 by a scale of at most 2^90 (which keeps the factors
      // finite where a channel is zero so far).  64 tokens of |v| <= vm add at most 8 vm to |S|; a loose bound costs
      // nothing until it is 2^15 times too large.  Lane: channels 2 lane, + 1, + 64, + 65.
      float bound[4];   // of the channels' states in 2-norm (the entering one's 1-norm: its squares may leave fp32)
      int field[4] = {300, 300, 300, 300};   // the scales' exponent fields
      float last[4] = {0.f, 0.f, 0.f, 0.f};  // the last chunk's largest |v|
      {
        const float *sums = reinterpret_cast<const float *>(sm + OFF_OUT);   // (until the first output)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int ch = 64 * (i >> 1) + 2 * lane + (i & 1);
          bound[i] = map ? 1.f : src ? (sums[ch] + sums[128 + ch]) + (sums[256 + ch] + sums[384 + ch]) : 0.f;
        }
      }
      for (int c = 0; c < nchunks; ++c) {
        const uint8_t *st = sm + (c & 1) * kStage;
        const int valid = min(kC, len - c * kC);
        wait_or_abort(&bar[B_VAL + (c & 1)], (c >> 1) & 1, s_abort, prm.status);
        uint32_t top[2] = {0u, 0u};   // |v|'s bits (bf16 order is integer order)
#pragma unroll 8
        for (int t = 0; t < valid; ++t) {
          const uint8_t *at = st + ST_V + swz_offset(64, t, 2 * lane);
          top[0] = __vmaxu2(top[0], *reinterpret_cast<const uint32_t *>(at) & 0x7FFF7FFFu);
          top[1] = __vmaxu2(top[1], *reinterpret_cast<const uint32_t *>(at + 8192) & 0x7FFF7FFFu);
        }
        // the last chunk's decay and growth (its block has long landed, and its stage is held until these scales are out)
        float gamma = 1.f;
        if (c > 0) {
          wait_or_abort(&bar[B_FULL + ((c - 1) & 1)], ((c - 1) >> 1) & 1, s_abort, prm.status);
          gamma = reinterpret_cast<const float *>(sm + ((c - 1) & 1) * kStage + ST_BLK + kBlkVec)[kVecGamma];
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float vm = i & 1 ? __uint_as_float(top[i >> 1] & 0xFFFF0000u) : __uint_as_float(top[i >> 1] << 16);
          bound[i] = fminf(fmaf(gamma, bound[i], 8.f * last[i]), 3.4e38f);   // (an infinite one would never fall again)
          last[i] = vm;
          const float most = fmaf(9.f, vm, bound[i]);
          // (kept until it is too large, or 2^10 too small)
          const int want = min(max(267 - static_cast<int>(__float_as_uint(most) >> 23 & 0xFF), 1), 217);
          if (want < field[i] || want > field[i] + 10) field[i] = want;
          const int ch = 128 * (c & 1) + 64 * (i >> 1) + 2 * lane + (i & 1);
          s_sig[ch] = __uint_as_float(static_cast<uint32_t>(field[i]) << 23);
          s_inv[ch] = __uint_as_float(static_cast<uint32_t>(254 - field[i]) << 23);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar[B_SCALE + (c & 1)]);   // (the workers wait for it, so their word that the stage is free
                                                         // is this warp's too)
      }
    } else if (!worker) {
      // ------------------------------------------------------------ products: this warp's accumulator of the pairs
      const int me = warp - kIssuer;
      constexpr uint32_t id1 = idesc_bf16(128, 64, false, false), id2 = idesc_f16(128, 64, false, false),
                         id3 = idesc_f16(128, 128, false, true), idv = idesc_bf16(128, 64, true, false);
      const uint64_t one = desc_kmajor_base(smem_u32(sm + OFF_ONE)), k16 = desc_mnmajor_base(smem_u32(sm + OFF_K16), 64);
      uint32_t longs = 0;   // chunks with long rows so far
      const uint32_t ku = tmem + TM_KU + 64 * me, uu = tmem + TM_U + 64 * me, sp = tmem + TM_S + 64 * me;
      for (int c = 0; c < nchunks; ++c) {
        uint8_t *st = sm + (c & 1) * kStage;
        const uint64_t kk = desc_kmajor_base(smem_u32(st)), qq = kk + desc_bytes(8192), vt = desc_mnmajor_base(smem_u32(st + ST_V), 64);
        const uint64_t l1 = desc_kmajor_base(smem_u32(st + ST_BLK)), pp = l1 + desc_bytes(kBlkP), l2 = l1 + desc_bytes(kBlkL2);
        auto values = [&] {
#pragma unroll
          for (int k = 0; k < 4; ++k) mma_bf16(tmem + TM_V, vt + mnmajor_step(k), one + kmajor_step(64, k), idv, k > 0);
          mma_commit(&bar[B_V]);
        };
        // (a ragged chunk's rows behind the end are cleared before S is announced; D before, which values run behind)
        const bool ragged = len - c * kC < kC;
        if (me == 1 && !ragged) {
          wait_or_abort(&bar[B_VAL + (c & 1)], (c >> 1) & 1, s_abort, prm.status);
          if (c > 0) wait_or_abort(&bar[B_M3], (c - 1) & 1, s_abort, prm.status);
          tc_fence_after();
          if (lane == 0) values();
          __syncwarp();
        }
        wait_or_abort(&bar[B_VAL + (c & 1)], (c >> 1) & 1, s_abort, prm.status);
        wait_or_abort(&bar[B_FULL + (c & 1)], (c >> 1) & 1, s_abort, prm.status);
        {   // long rows, scaled as they were for the block (this warp's: keys or queries; both warps' products read both)
          const uint32_t *rows = reinterpret_cast<const uint32_t *>(st + ST_BLK + kBlkVec) + kVecLong;
          const uint4 rows4 = *reinterpret_cast<const uint4 *>(rows);
          if (rows4.x | rows4.y | rows4.z | rows4.w) {
            for (int half = 0; half < 2; ++half)
              if (rows[2 * me + half] >> lane & 1)
                for (int ch = 0; ch < kD; ch += 8) scale_piece(st + swz_offset(128, 64 * me + 32 * half + lane, ch));
            fence_async_smem();
            warp_arrive(&bar[B_LONG]);
            wait_or_abort(&bar[B_LONG], longs++ & 1, s_abort, prm.status);
          }
        }
        wait_or_abort(&bar[B_S], c & 1, s_abort, prm.status);   // S is in place, D has been read
        tc_fence_after();
        if (lane == 0) {
          if (me == 1 && ragged) values();
#pragma unroll
          for (int k = 0; k < 8; ++k) mma_bf16_tmem_a(ku, sp + 8 * k, kk + kmajor_step(128, k), id1, k > 0);
          mma_commit(&bar[B_M1]);
          if (me == 1 && known) {
#pragma unroll
            for (int k = 0; k < 8; ++k)
              mma_bf16_tmem_a(tmem + TM_QS, tmem + TM_S + 8 * k, qq + kmajor_step(128, k), id1, k > 0);
          }
        }
        __syncwarp();
        wait_or_abort(&bar[B_R], c & 1, s_abort, prm.status);   // R is in place, KU and VT have been read
        tc_fence_after();
        if (lane == 0) {
          if (me == 0) {   // R hi L hi, and half of R hi L lo
#pragma unroll
            for (int k = 0; k < 4; ++k) mma_bf16_tmem_a(uu, tmem + TM_R + 8 * k, l1 + kmajor_step(64, k), id2, k > 0);
#pragma unroll
            for (int k = 0; k < 2; ++k) mma_bf16_tmem_a(uu, tmem + TM_R + 8 * k, l2 + kmajor_step(64, k), id2, 1);
          } else {         // R lo L hi, and the other half
#pragma unroll
            for (int k = 0; k < 4; ++k) mma_bf16_tmem_a(uu, tmem + TM_R + 32 + 8 * k, l1 + kmajor_step(64, k), id2, k > 0);
#pragma unroll
            for (int k = 2; k < 4; ++k) mma_bf16_tmem_a(uu, tmem + TM_R + 8 * k, l2 + kmajor_step(64, k), id2, 1);
          }
          mma_commit(&bar[B_M2]);
        }
        __syncwarp();
        wait_or_abort(&bar[B_U], c & 1, s_abort, prm.status);   // U, U', the fp16 keys are in place, the accumulators read
        tc_fence_after();
        if (me == 0 && lane == 0) {
          if (known) {
#pragma unroll
            for (int k = 0; k < 4; ++k) mma_bf16_tmem_a(tmem + TM_OT, tmem + TM_UH + 8 * k, pp + kmajor_step(64, k), id2, k > 0);
            mma_commit(&bar[B_O]);
          }
#pragma unroll
          for (int p = 0; p < 2; ++p)
#pragma unroll
            for (int k = 0; k < 4; ++k)
              mma_bf16_tmem_a(tmem + TM_D, tmem + TM_R + 32 * p + 8 * k, k16 + mnmajor_step(k), id3, p + k > 0);
          mma_commit(&bar[B_M3]);
        }
        __syncwarp();
      }
    } else {
      // ------------------------------------------------------------ epilogues
      const uint32_t lanes = tmem + (static_cast<uint32_t>(quad * 32) << 16);
      // this quarter of S -> its two parts, ahead of chunk c; v's rows behind a ragged chunk's end, which may hold
      // anything, are cleared (0 x NaN is not 0; the fp16 keys there become 0)
      auto store_s = [&](int c) {
        const int valid = len - c * kC;
        if (valid < kC) {
          wait_or_abort(&bar[B_VAL + (c & 1)], (c >> 1) & 1, s_abort, prm.status);
          for (int i = tid; i < (kC - valid) * 16; i += kWorkers)
            *reinterpret_cast<uint4 *>(sm + (c & 1) * kStage + ST_V + swz_offset(64, valid + (i >> 4), 8 * (i & 15))) =
                make_uint4(0, 0, 0, 0);
          fence_async_smem();
        }
        uint32_t p1[16], p2[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) split2(make_float2(S[2 * i], S[2 * i + 1]), p1[i], p2[i]);
        tmem_st16(lanes + TM_S + 16 * cg, p1);
        tmem_st16(lanes + TM_S + 64 + 16 * cg, p2);
        tmem_wait_st();
        tc_fence_before();
        warp_arrive(&bar[B_S]);
      };
      auto store_r = [&](const float2 (&x)[8], int which) {   // 16 tokens of R or U' -> their two parts
        uint32_t p1[8], p2[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) split2h(x[i], p1[i], p2[i]);
        tmem_st8(lanes + TM_R + 8 * cg, p1);
        tmem_st8(lanes + TM_R + 32 + 8 * cg, p2);
        tmem_wait_st();
        tc_fence_before();
        warp_arrive(&bar[which]);
      };
      // S is kept times its channel's scale: announced with chunk 0's, and brought to the next chunk's where that differs
      wait_or_abort(&bar[B_SCALE], 0, s_abort, prm.status);
      float sig = s_sig[d];
#pragma unroll
      for (int e = 0; e < 32; ++e) S[e] *= sig;
      store_s(0);
      for (int c = 0; c < nchunks; ++c) {
        uint8_t *st = sm + (c & 1) * kStage;
        const float *vec = reinterpret_cast<const float *>(st + ST_BLK + kBlkVec);
        const int valid = min(kC, len - c * kC);
        wait_or_abort(&bar[B_FULL + (c & 1)], (c >> 1) & 1, s_abort, prm.status);
        // ---- under the product: v^T (this thread's channel of 16 tokens)
        float2 x[8];
        const float gamma = vec[kVecGamma];
        const float2 sig2 = make_float2(sig, sig);
        {   // R^T = beta (v^T - e^b/|k| (k S)^T)
          uint32_t w[16], w2[16];
          wait_or_abort(&bar[B_V], c & 1, s_abort, prm.status);
          tc_fence_after();
          tmem_ld16_async(lanes + TM_V + 16 * cg, w);
          tmem_wait_ld();
          tmem_tie<16>(w);
#pragma unroll
          for (int i = 0; i < 8; i += 2) {
            const float4 b = *reinterpret_cast<const float4 *>(vec + kVecB + 16 * cg + 2 * i);
            x[i] = mul2(mul2(make_float2(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1])), sig2), make_float2(b.x, b.y));
            x[i + 1] = mul2(mul2(make_float2(__uint_as_float(w[2 * i + 2]), __uint_as_float(w[2 * i + 3])), sig2), make_float2(b.z, b.w));
          }
          wait_or_abort(&bar[B_M1], c & 1, s_abort, prm.status);
          tc_fence_after();
          tmem_ld16_async(lanes + TM_KU + 16 * cg, w);
          tmem_ld16_async(lanes + TM_KU + 64 + 16 * cg, w2);
          tmem_wait_ld();
          tmem_tie<16>(w);
          tmem_tie<16>(w2);
#pragma unroll
          for (int i = 0; i < 8; i += 2) {
            const float4 k = *reinterpret_cast<const float4 *>(vec + kVecK + 16 * cg + 2 * i);
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              const int j = i + y;
              const float2 ku = add2(make_float2(__uint_as_float(w[2 * j]), __uint_as_float(w[2 * j + 1])),
                                     make_float2(__uint_as_float(w2[2 * j]), __uint_as_float(w2[2 * j + 1])));
              x[j] = fma2(y ? make_float2(k.z, k.w) : make_float2(k.x, k.y), ku, x[j]);
            }
          }
          if (valid < kC) {   // k S there may be anything
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              if (16 * cg + 2 * i >= valid) x[i].x = 0.f;
              if (16 * cg + 2 * i + 1 >= valid) x[i].y = 0.f;
            }
          }
          store_r(x, B_R);
        }
        // ---- under U: the chunk's keys times 2^-x as fp16 (thread: row tid / 8, two pieces of 8 channels); rows behind
        // the end are 0
        {
          const int r = tid >> 3, c0 = 8 * (tid & 7);
          const float f = vec[kVecX + r];
#pragma unroll
          for (int y = 0; y < 128; y += 64) {
            uint4 w = *reinterpret_cast<const uint4 *>(st + swz_offset(128, r, c0 + y));
            const float2 f2 = make_float2(f, f);
            w.x = pack_f16x2(mul2(unpack_bf16x2(w.x), f2));
            w.y = pack_f16x2(mul2(unpack_bf16x2(w.y), f2));
            w.z = pack_f16x2(mul2(unpack_bf16x2(w.z), f2));
            w.w = pack_f16x2(mul2(unpack_bf16x2(w.w), f2));
            if (r >= valid) w = make_uint4(0, 0, 0, 0);
            *reinterpret_cast<uint4 *>(sm + OFF_K16 + swz_offset(64, r, c0 + y)) = w;
          }
          fence_async_smem();
        }
        {   // U^T = (L R)^T, its first part;  U'^T = 2^x e^(b_63 - b)/|k| U^T
          uint32_t w[16], w2[16], uh[8];
          wait_or_abort(&bar[B_M2], c & 1, s_abort, prm.status);
          tc_fence_after();
          tmem_ld16_async(lanes + TM_U + 16 * cg, w);
          tmem_ld16_async(lanes + TM_U + 64 + 16 * cg, w2);
#pragma unroll
          for (int i = 0; i < 8; i += 2) {
            const float4 f = *reinterpret_cast<const float4 *>(vec + kVecS + 16 * cg + 2 * i);
            x[i] = make_float2(f.x, f.y);
            x[i + 1] = make_float2(f.z, f.w);
          }
          tmem_wait_ld();
          tmem_tie<16>(w);
          tmem_tie<16>(w2);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float2 u = add2(make_float2(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1])),
                                  make_float2(__uint_as_float(w2[2 * i]), __uint_as_float(w2[2 * i + 1])));
            uh[i] = pack_f16x2(u);
            x[i] = mul2(x[i], u);
          }
          if (known) tmem_st8(lanes + TM_UH + 8 * cg, uh);
          store_r(x, B_U);
        }
        if (known) {   // beside the state's product: o^T = scale e^b/|q| (q S)^T + scale (P U)^T.  Here a thread holds the fragments
            // that stmatrix transposes: channels lane / 4 + 8 i, tokens 2 (lane % 4), + 1 (+ 8) of the warp's 32 x 16
          if (c > 0) wait_or_abort(&bar[B_OUT], (c - 1) & 1, s_abort, prm.status);   // the tile is free
          const float *si = s_inv + 128 * (c & 1) + 32 * quad + (lane >> 2);
          const float inv4[4] = {si[0], si[8], si[16], si[24]};
          const uint32_t ot = smem_u32(sm + OFF_OUT + 8192 * (quad >> 1));
          const float2 f0 = *reinterpret_cast<const float2 *>(vec + kVecQ + 16 * cg + 2 * (lane & 3));
          const float2 f1 = *reinterpret_cast<const float2 *>(vec + kVecQ + 16 * cg + 2 * (lane & 3) + 8);
          wait_or_abort(&bar[B_O], c & 1, s_abort, prm.status);
          tc_fence_after();
          uint32_t w[16], y[16];
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {
            tmem_ld_frag(lanes + (static_cast<uint32_t>(16 * hf) << 16) + TM_QS + 16 * cg, w + 8 * hf);
            tmem_ld_frag(lanes + (static_cast<uint32_t>(16 * hf) << 16) + TM_OT + 16 * cg, y + 8 * hf);
          }
          tmem_wait_ld();
          tmem_tie<16>(w);
          tmem_tie<16>(y);
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {   // 16 channels
            const float2 s0 = make_float2(inv4[2 * hf], inv4[2 * hf]), s1 = make_float2(inv4[2 * hf + 1], inv4[2 * hf + 1]);
            uint32_t p[4];   // (channels 0..7, tokens 0..7), (8..15, 0..7), (0..7, 8..15), (8..15, 8..15)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float2 q = make_float2(__uint_as_float(w[8 * hf + 2 * i]), __uint_as_float(w[8 * hf + 2 * i + 1]));
              const float2 u = make_float2(__uint_as_float(y[8 * hf + 2 * i]), __uint_as_float(y[8 * hf + 2 * i + 1]));
              p[i] = pack2(mul2(i & 1 ? s1 : s0, fma2(i & 2 ? f1 : f0, q, mul2(make_float2(prm.scale, prm.scale), u))));
            }
            // lane: the address of token (lane & 7) + 8 (lane >> 4), channels 16 hf + 8 ((lane >> 3) & 1) ..
            const int tk = 16 * cg + (lane & 7) + 8 * (lane >> 4), ch = 32 * (quad & 1) + 16 * hf + (lane & 8);
            asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};"
                         ::"r"(ot + swz_offset(64, tk, ch)), "r"(p[0]), "r"(p[1]), "r"(p[2]), "r"(p[3])
                         : "memory");
          }
          fence_async_smem();
          warp_arrive(&bar[B_TILE]);
        }
        {   // S = e^(b_63) S + D, ready for the next chunk's scale
          uint32_t w[32];
          const float2 g2 = make_float2(gamma, gamma);
          float ratio = 1.f;
          if (c + 1 < nchunks) {
            wait_or_abort(&bar[B_SCALE + ((c + 1) & 1)], ((c + 1) >> 1) & 1, s_abort, prm.status);
            const float next = s_sig[128 * ((c + 1) & 1) + d];
            ratio = next * s_inv[128 * (c & 1) + d];   // a power of two, nearly always 1
            sig = next;
          }
          wait_or_abort(&bar[B_M3], c & 1, s_abort, prm.status);
          tc_fence_after();
          tmem_ld16_async(lanes + TM_D + 32 * cg, w);
          tmem_ld16_async(lanes + TM_D + 32 * cg + 16, w + 16);
          tmem_wait_ld();
          tmem_tie<32>(w);
#pragma unroll
          for (int i = 0; i < 32; i += 2) {
            const float2 y = fma2(g2, make_float2(S[i], S[i + 1]), make_float2(__uint_as_float(w[i]), __uint_as_float(w[i + 1])));
            S[i] = y.x;
            S[i + 1] = y.y;
          }
          if (__any_sync(0xffffffffu, ratio != 1.f)) {
#pragma unroll
            for (int i = 0; i < 32; ++i) S[i] *= ratio;
          }
          if (c + 1 < nchunks) store_s(c + 1);
          if (SEGMENTS && mid && c + 1 == job.mid_chunk && c + 1 < nchunks) {
            const float inv = s_inv[128 * ((c + 1) & 1) + d];
#pragma unroll
            for (int e = 0; e < 32; ++e) mid[(32 * cg + e) * kD + d] = S[e] * inv;
          }
        }
        warp_arrive(&bar[B_FREE]);   // the last read of the stage is behind
      }
      const float inv = s_inv[128 * ((nchunks - 1) & 1) + d];
#pragma unroll
      for (int e = 0; e < 32; ++e) S[e] *= inv;
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kProducer) {
      tc_fence_after();
      tmem_dealloc(tmem, kTmemCols);
    }
  }
  if (nchunks == 0 && tid == 0) grid_dependency_wait();
  if (worker && dst) {
#pragma unroll
    for (int e = 0; e < 32; ++e) dst[(32 * cg + e) * kD + d] = S[e];
  }
}

// Entering states, S' = F S + B (S' goes where B is), in fp32, a sequence's (`chunks` of them) one behind the other from S
// (matrix src; F: mid .., B: dst ..), or alone: a CTA per job, head and 16 value channels.  F comes to shared memory, the
// next one during a step (where there is one).  A thread sums half of the key channels for two rows and 8 value channels,
// two products an instruction; the halves meet in shared memory.  Bound by the issue of a step's products and operand
// reads (1400 cycles) and the latency around them.
namespace jn {
constexpr int kParts = 8, kThreads = 256, kStride = 132;   // value channels / 16; floats of a row of F
constexpr uint32_t kF = kD * kStride * 4, OFF_S = 0, OFF_SUM = 2 * kD * 64, OFF_F = 3 * kD * 64;   // S: two of [128][16]
constexpr uint32_t smem_bytes(int steps) { return OFF_F + (steps > 1 ? 2 : 1) * kF; }
}  // namespace jn
__global__ void __launch_bounds__(jn::kThreads) gdn_join_kernel(const __grid_constant__ GdnPrefillParams prm) {
  using namespace jn;
  extern __shared__ __align__(16) uint8_t smem_raw[];
  const int tid = threadIdx.x, part = blockIdx.x % kParts, h = blockIdx.x / kParts % prm.Hv;
  const GdnJob job = prm.job[blockIdx.x / kParts / prm.Hv];
  const auto mat = [&](int m) { return prm.mats + (static_cast<size_t>(m) * prm.Hv + h) * kD * kD; };
  float *const s_state = reinterpret_cast<float *>(smem_raw + OFF_S), *const s_sum = reinterpret_cast<float *>(smem_raw + OFF_SUM);
  const auto fetch = [&](int j) {
    const float *src = mat(job.mid + j);
    const uint32_t dst = smem_u32(smem_raw) + OFF_F + (j & 1) * kF;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const int x = i * kThreads + tid;   // 16 bytes: row x / 32, piece x % 32
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst + (x >> 5) * kStride * 4 + (x & 31) * 16), "l"(src + 4 * x) : "memory");
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  grid_dependency_wait();
  fetch(0);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int x = i * kThreads + tid;     // 16 bytes: row x / 4, piece x % 4
    *reinterpret_cast<float4 *>(s_state + 4 * x) = *reinterpret_cast<const float4 *>(mat(job.src) + (x >> 2) * kD + 16 * part + 4 * (x & 3));
  }
  const int k0 = tid >> 7 ? kD / 2 : 0, c0 = 8 * (tid & 1), row = (tid & 127) >> 1;   // and row + 64
  for (int j = 0; j < job.chunks; ++j) {
    const bool more = j + 1 < job.chunks;
    if (more) fetch(j + 1);
    float *out = mat(job.dst + j) + row * kD + 16 * part + c0;
    float4 b[2][2];
    if (k0 == 0) {
#pragma unroll
      for (int r = 0; r < 2; ++r)
#pragma unroll
        for (int x = 0; x < 2; ++x) b[r][x] = *reinterpret_cast<const float4 *>(out + r * 64 * kD + 4 * x);
    }
    if (more) asm volatile("cp.async.wait_group 1;" ::: "memory");
    else asm volatile("cp.async.wait_group 0;" ::: "memory");
    __syncthreads();
    const float *f = reinterpret_cast<const float *>(smem_raw + OFF_F + (j & 1) * kF) + row * kStride + k0;
    const float *st = s_state + (j & 1) * kD * 16 + k0 * 16 + c0;
    float2 acc[2][4];
#pragma unroll
    for (int r = 0; r < 2; ++r)
#pragma unroll
      for (int x = 0; x < 4; ++x) acc[r][x] = make_float2(0.f, 0.f);
#pragma unroll 4
    for (int k = 0; k < kD / 2; k += 4) {
      const float4 fa = *reinterpret_cast<const float4 *>(f + k), fb = *reinterpret_cast<const float4 *>(f + 64 * kStride + k);
      const float a4[4] = {fa.x, fa.y, fa.z, fa.w}, b4[4] = {fb.x, fb.y, fb.z, fb.w};
#pragma unroll
      for (int kk = 0; kk < 4; ++kk) {
        const float4 s0 = *reinterpret_cast<const float4 *>(st + (k + kk) * 16), s1 = *reinterpret_cast<const float4 *>(st + (k + kk) * 16 + 4);
        const float2 s2[4] = {make_float2(s0.x, s0.y), make_float2(s0.z, s0.w), make_float2(s1.x, s1.y), make_float2(s1.z, s1.w)};
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          acc[0][x] = fma2(make_float2(a4[kk], a4[kk]), s2[x], acc[0][x]);
          acc[1][x] = fma2(make_float2(b4[kk], b4[kk]), s2[x], acc[1][x]);
        }
      }
    }
    float *sum = s_sum + row * 16 + c0;
    if (k0 != 0) {
#pragma unroll
      for (int r = 0; r < 2; ++r)
#pragma unroll
        for (int x = 0; x < 2; ++x)
          *reinterpret_cast<float4 *>(sum + r * 64 * 16 + 4 * x) = make_float4(acc[r][2 * x].x, acc[r][2 * x].y, acc[r][2 * x + 1].x, acc[r][2 * x + 1].y);
    }
    __syncthreads();
    if (k0 == 0) {
      float *next = s_state + ((j + 1) & 1) * kD * 16 + row * 16 + c0;
#pragma unroll
      for (int r = 0; r < 2; ++r)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const float4 u = *reinterpret_cast<const float4 *>(sum + r * 64 * 16 + 4 * x);
          const float4 y = make_float4(acc[r][2 * x].x + u.x + b[r][x].x, acc[r][2 * x].y + u.y + b[r][x].y,
                                       acc[r][2 * x + 1].x + u.z + b[r][x].z, acc[r][2 * x + 1].y + u.w + b[r][x].w);
          *reinterpret_cast<float4 *>(next + r * 64 * 16 + 4 * x) = y;
          *reinterpret_cast<float4 *>(out + r * 64 * kD + 4 * x) = y;
        }
    }
    __syncthreads();   // (F's buffer and the sums are free, the next state is in place)
  }
}

int chunks_of(const GdnPrefillParams &p, int n) { return (p.cu[n + 1] - p.cu[n] + kC - 1) / kC; }

// Segments of a sequence: a first one of g chunks, inner ones of as many, and a last one of 1 to g.
struct Cut {
  int g = 0, halves = 1;   // chunks of a segment (0: sequences stay whole), pieces of an inner one in the second grid
  bool whole(int chunks) const { return chunks <= g; }
  int half() const { return (g + 1) / 2; }
  int inner(int chunks) const { return (chunks + g - 1) / g - 2; }
  int last(int chunks) const { return chunks - (inner(chunks) + 1) * g; }
  int matrices(int chunks) const { return 1 + (halves == 2 ? 4 : 2) * inner(chunks); }
};

// How to cut, by estimates in chunks' time.  A grid of at most one CTA per SM takes its longest piece; others are bounded
// (from below for whole sequences, from above for segments).
Cut choose_cut(const GdnPrefillParams &p, int max_mats) {
  const int longest = chunks_of(p, p.order[0]);
  int64_t sum = 0;
  Cut best_cut;
  if (longest < kSegmentExtra + 2 * kSegmentMin || p.num_seqs > kGdnMaxJobs) return best_cut;
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess ||
      sms <= 0)
    sms = 152;
  for (int n = 0; n < p.num_seqs; ++n) sum += chunks_of(p, n);
  int64_t best = std::max<int64_t>(longest, sum * p.Hv / sms);
  if (sum * p.Hv / sms + kSegmentExtra >= longest) return best_cut;   // the work alone takes as long
  for (int m = 2; m <= kGdnMaxSegs; ++m)
    for (int halves = 1; halves <= 2; ++halves) {
      Cut cut;
      cut.halves = halves;
      cut.g = halves == 1 ? (longest + m - 1) / m : (2 * longest + 2 * m - 2) / (2 * m - 1);
      if (cut.g < kSegmentMin * halves) continue;
      int64_t jobs1 = 0, jobs2 = 0, work1 = 0, work2 = 0, mats = 0;
      int piece = 0;
      for (int n = 0; n < p.num_seqs; ++n) {
        const int chunks = chunks_of(p, n);
        if (cut.whole(chunks)) {
          jobs1 += 1;
          work1 += chunks;
          continue;
        }
        const int k = cut.inner(chunks);
        jobs1 += 1 + 2 * k;
        work1 += static_cast<int64_t>(1 + 2 * k) * cut.g;
        jobs2 += 1 + k * halves;
        work2 += chunks - cut.g;
        mats += cut.matrices(chunks);
        piece = std::max({piece, cut.last(chunks), k == 0 ? 0 : halves == 2 ? cut.half() : cut.g});
      }
      if (jobs1 > kGdnMaxJobs || jobs2 > kGdnMaxJobs || mats * p.Hv > max_mats) continue;
      const auto grid = [&](int64_t jobs, int64_t work, int longest_piece) {
        return jobs * p.Hv <= sms ? longest_piece : work * p.Hv / sms + longest_piece + kWaveExtra * (jobs * p.Hv / sms);
      };
      const int64_t est = grid(jobs1, work1, cut.g) + grid(jobs2, work2, piece) + kSegmentExtra + (halves == 2 ? kHalvesExtra : 0);
      if (est < best) {
        best = est;
        best_cut = cut;
      }
    }
  return best_cut;
}

cudaError_t launch_segments(GdnPrefillParams &p, const Cut &cut, float *mats, cudaStream_t stream) {
  const int g = cut.g, half = cut.half();
  p.mats = mats;
  int jobs = 0;
  const auto add = [&](int i, int src, int dst, int chunk0, int chunks, int mid = -1) {
    p.job[jobs++] = {p.order[i], static_cast<int16_t>(src), static_cast<int16_t>(dst), static_cast<int16_t>(mid), chunk0, chunks, half};
  };
  // every sequence that is cut (they come longest first), with its inner segments and its first matrix
  const auto each = [&](auto body) {
    int base = 0;
    for (int i = 0; i < p.num_seqs && !cut.whole(chunks_of(p, p.order[i])); ++i) {
      const int chunks = chunks_of(p, p.order[i]), k = cut.inner(chunks);
      body(i, chunks, k, base, base + k + 1 /* F */, base + 2 * k + 1 /* half way: B, S */, base + 3 * k + 1 /* F */);
      base += cut.matrices(chunks);
    }
  };
  const auto run = [&](auto kernel, int per_head, int threads, size_t smem) {
    const int n = jobs;
    jobs = 0;
    return n ? launch_dependent(kernel, n * p.Hv * per_head, threads, smem, stream, p) : cudaSuccess;
  };
  // first segments, F and B of the inner ones, then the sequences that stay whole
  each([&](int i, int, int, int base, int, int, int) { add(i, kFromCaller, base, 0, g); });
  each([&](int i, int, int k, int base, int f, int mb, int mf) {
    for (int j = 0; j < k; ++j) {
      add(i, kFromZero, base + 1 + j, (1 + j) * g, g, cut.halves == 2 ? mb + j : -1);
      add(i, kFromIdentity, f + j, (1 + j) * g, g, cut.halves == 2 ? mf + j : -1);
    }
  });
  for (int i = 0; i < p.num_seqs; ++i) {
    const int chunks = chunks_of(p, p.order[i]);
    if (cut.whole(chunks)) add(i, kFromCaller, kToCaller, 0, chunks);
  }
  p.behind = 0;
  if (const cudaError_t e = run(gdn_chain_kernel<true>, 1, ch::kThreads, ch::kSmemBytes)) return e;
  // entering states, then the half-way ones from them
  each([&](int i, int, int k, int base, int f, int, int) {
    if (k) add(i, base, base + 1, 0, k, f);
  });
  if (const cudaError_t e = run(gdn_join_kernel, jn::kParts, jn::kThreads, jn::smem_bytes(2))) return e;
  if (cut.halves == 2) {
    each([&](int i, int, int k, int base, int, int mb, int mf) {
      for (int j = 0; j < k; ++j) add(i, base + j, mb + j, 0, 1, mf + j);
    });
    if (const cudaError_t e = run(gdn_join_kernel, jn::kParts, jn::kThreads, jn::smem_bytes(1))) return e;
  }
  each([&](int i, int chunks, int k, int base, int, int mb, int) {
    add(i, base + k, kToCaller, (1 + k) * g, chunks - (1 + k) * g);
    for (int j = 0; j < k; ++j) {
      add(i, base + j, kToNothing, (1 + j) * g, cut.halves == 2 ? half : g);
      if (cut.halves == 2) add(i, mb + j, kToNothing, (1 + j) * g + half, g - half);
    }
  });
  p.behind = 1;
  return run(gdn_chain_kernel<true>, 1, ch::kThreads, ch::kSmemBytes);
}

}  // namespace

namespace {
// matrices (times heads) that a batch of so many tokens has room for: a segment has kSegmentMin chunks or more, in halves
// twice as many, and 2 matrices, in halves 4; none where no sequence can be long enough
int64_t matrix_room(int64_t total_tokens, int Hv) {
  const int64_t chunks = total_tokens / kC + 1;
  if (chunks < kSegmentExtra + 2 * kSegmentMin) return 0;
  return std::min<int64_t>(kGdnMaxMats, 2 * chunks / kSegmentMin * Hv);
}
size_t block_bytes(int64_t total_tokens, int num_seqs, int Hv) {
  return (total_tokens / kC + num_seqs) * static_cast<size_t>(Hv) * kGdnBlkBytes;
}
}  // namespace

size_t gdn_prefill_workspace_bytes(int64_t total_tokens, int num_seqs, int Hv) {
  return block_bytes(total_tokens, num_seqs, Hv) + matrix_room(total_tokens, Hv) * sizeof(float) * kD * kD;
}

cudaError_t launch_gdn_prefill(const GdnRecurrentArgs &a, const int32_t *cu_host, int num_seqs, uint8_t *blocks,
                               cudaStream_t stream) {
  static std::mutex mu;
  static uint64_t done = 0;
  if (const cudaError_t e = set_attributes_once(mu, done, [] {
        cudaError_t r = cudaFuncSetAttribute(gdn_intra_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, in::kSmemBytes);
        if (r == cudaSuccess)
          r = cudaFuncSetAttribute(gdn_chain_kernel<false>, cudaFuncAttributeMaxDynamicSharedMemorySize, ch::kSmemBytes);
        if (r == cudaSuccess)
          r = cudaFuncSetAttribute(gdn_chain_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize, ch::kSmemBytes);
        if (r == cudaSuccess)
          r = cudaFuncSetAttribute(gdn_join_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, jn::smem_bytes(2));
        return r;
      }))
    return e;
  GdnPrefillParams p;
  const int total = cu_host[num_seqs], Hk = a.Hv / a.group;
  const int room = static_cast<int>(matrix_room(total, a.Hv));
  float *mats = reinterpret_cast<float *>(blocks + block_bytes(total, num_seqs, a.Hv));
  if (!make_tokens_map(&p.tq, a.q, Hk, total, a.qk_stride) || !make_tokens_map(&p.tk, a.k, Hk, total, a.qk_stride) ||
      !make_tokens_map(&p.tv, a.v, a.Hv, total, a.v_stride) || !make_tokens_map(&p.tout, a.out, a.Hv, total, a.out_stride))
    return cudaErrorInvalidValue;
  p.a = a.a; p.beta = a.beta;
  p.a_stride = a.a_stride; p.beta_stride = a.beta_stride;
  p.A_log = a.A_log; p.dt_bias = a.dt_bias;
  p.scale = a.scale;
  p.Hk = Hk; p.Hv = a.Hv; p.group = a.group;
  p.num_slots = a.num_slots;
  p.state_in = a.state_in;
  p.state_out_pool = a.state_out_pool;
  p.out = a.out;
  p.out_stride = a.out_stride;
  p.status = a.status;
  for (int s0 = 0; s0 < num_seqs; s0 += kGdnMaxSeqs) {
    const int ns = std::min(kGdnMaxSeqs, num_seqs - s0);
    p.num_seqs = ns;
    p.slot_ids = a.slot_ids ? a.slot_ids + s0 : nullptr;
    p.state_out_dense = a.state_out_dense ? a.state_out_dense + static_cast<size_t>(s0) * a.Hv * kD * kD : nullptr;
    std::copy(cu_host + s0, cu_host + s0 + ns + 1, p.cu);
    std::iota(p.order, p.order + ns, uint16_t(0));
    std::stable_sort(p.order, p.order + ns, [&](int x, int y) { return p.cu[x + 1] - p.cu[x] > p.cu[y + 1] - p.cu[y]; });
    const int slots = (p.cu[ns] - p.cu[0]) / kC + ns;
    p.blocks = blocks;
    blocks += static_cast<size_t>(slots) * a.Hv * kGdnBlkBytes;
    if (const cudaError_t e = launch_dependent(gdn_intra_kernel, static_cast<unsigned>(slots) * Hk, in::kThreads, in::kSmemBytes,
                                               stream, p))
      return e;
    const Cut cut = choose_cut(p, room);
    if (const cudaError_t e = cut.g ? launch_segments(p, cut, mats, stream) : launch_dependent(gdn_chain_kernel<false>, ns * a.Hv, ch::kThreads, ch::kSmemBytes, stream, p)) return e;
  }
  return cudaSuccess;
}

}  // namespace kda
