// Chunked prefill of the gated delta rule on sm_103a.
//
// With chunks of C = 64 tokens, b_t the cumulative log-decay inside a chunk, k^, q^ the l2-normalised keys and
// queries and S the state entering the chunk, the recurrence S_t = (I - beta k^ k^T) e^lambda S_{t-1} + beta k^ v^T is
//
//   A_ri = beta_r k^_r.k^_i e^(b_r - b_i)  (i < r),     T = (I + A)^-1 Diag(beta)
//   P_ri = scale q^_r.k^_i e^(b_r - b_i)   (i <= r)
//   R_i  = v_i - e^(b_i) S^T k^_i,   U = T R
//   o_r  = scale e^(b_r) S^T q^_r + (P T R)_r,   S' = e^(b_63) S + sum_i e^(b_63 - b_i) k^_i U_i^T
//
// The decay is one number per token, so every product runs on the caller's own bf16 keys and queries and the norms
// and decays are fp32 factors of rows and columns: nothing is rounded that the caller did not round.
//
// Two kernels.  The intra-chunk kernel forms T and P T of every (chunk, value head) at once: 25 KB a block instead of
// the keys' and queries' decayed copies.  The state pass walks a sequence's chunks with S in fp32 registers, three
// products a chunk.  Where a product's operand is not the caller's data (S, T, R, the scaled U) it is a pair of bf16,
// hi + lo (16 bits of mantissa): hi and lo stand side by side as one N = 128 operand, so the second half costs one
// longer instruction and no second pass over the A operand.  A state then carries a relative error of a few 1e-6
// (single bf16 operands: a few 1e-3), as fp32 storage of it deserves.
#include <cuda.h>

#include <algorithm>
#include <numeric>
#include <vector>

#include "kda_common.cuh"
#include "kda_internal.h"
#include "kda_sm100.cuh"

namespace kda {
namespace {

using namespace sm100;

constexpr int kC = 64;
// a block: [T hi ; P T] (128 rows x 64 tokens, bf16, 128-byte row swizzle) | T lo (64 rows) | factors
constexpr uint32_t kBlkTlo = 16384, kBlkVec = 24576;
constexpr uint32_t kGdnBlkBytes = 25600;
// factors (fp32): e^(b_i) |k_i|^-1 | scale e^(b_r) |q_r|^-1 | e^(b_63 - b_i) |k_i|^-1 | e^(b_63)
constexpr int kVecK = 0, kVecQ = 64, kVecS = 128, kVecGamma = 192;
constexpr int kGdnMaxSeqs = 1024;   // sequences per launch (longer batches are split on the host)

struct GdnPrefillParams {
  CUtensorMap tq, tk, tv;       // [tokens, H, 128] bf16, box 64 channels x 1 head x 64 tokens, 128-byte swizzle
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
};
static_assert(sizeof(GdnPrefillParams) <= 32764, "kernel parameters are limited to 32764 bytes");

// Chunk slots: sequence n's chunks start at slot cu[n] / 64 + n (relative to the launch's first token), which leaves
// each sequence its ceil(len / 64) slots whatever the lengths are.
__host__ __device__ __forceinline__ int first_slot(const GdnPrefillParams &p, int n) { return (p.cu[n] - p.cu[0]) / kC + n; }

__device__ __forceinline__ void wait_or_abort(uint64_t *bar, uint32_t parity, volatile uint32_t *abort_flag,
                                              uint32_t *status) {
  if (*abort_flag) return;
  if (!mbar_wait(bar, parity)) {
    *abort_flag = 1;
    atomicOr(status, KDA_DEVICE_TIMEOUT);
  }
}

// x as a pair of bf16, hi + lo, of two neighbouring values
__device__ __forceinline__ void split2(float x, float y, uint32_t &hi, uint32_t &lo) {
  hi = pack_bf16x2(x, y);
  const float2 h = unpack_bf16x2(hi);
  lo = pack_bf16x2(x - h.x, y - h.y);
}

// ================================================================ intra-chunk kernel
namespace in {
constexpr int kThreads = 256;   // 8 warps; three CTAs per SM
constexpr uint32_t OFF_KQ = 0;  // [k ; q], 128 rows x 128 channels: consumed by the first product
constexpr int kStride = 68;
constexpr uint32_t OFF_A = 0;                          // A fp32 [64][68], turned into (I + A)^-1 in place
constexpr uint32_t OFF_P = 64 * kStride * 4;           // P fp32 [64][68]
constexpr uint32_t OFF_BLK = 35840;                    // the block's image
constexpr uint32_t OFF_SMALL = OFF_BLK + kGdnBlkBytes;
constexpr uint32_t SM_NORM = 0 /* [128]: 1 / |k_r|, 1 / |q_r| */, SM_BETA = 512, SM_BI = 768, SM_BF = 1024 /* b, whole and
                   fractional part */, SM_BAR = 1280, SM_TMEM = 1296, SM_ABORT = 1300, SM_END = 1312;
constexpr uint32_t kSmemBytes = OFF_SMALL + SM_END + 1024;
static_assert(OFF_BLK >= 2 * 64 * kStride * 4 && OFF_BLK >= 32768 && OFF_BLK % 1024 == 0, "shared memory map");
static_assert(3 * (kSmemBytes + 1024) <= 233472, "three CTAs per SM");
constexpr uint32_t kTmemCols = 128;
}  // namespace in

// 16 x 8 tile += X Y for X (16 x 8 ks), Y (8 ks x 8), fp32 with row stride in::kStride, on TF32 tensor cores; kExact: each
// operand as a pair of TF32 (three products: the error falls from 2^-11 to about 2^-21)
template <bool kExact>
__device__ __forceinline__ void mm_tile(float (&d)[4], const float *X, const float *Y, int ks, int lane) {
  const int g = lane >> 2, t = lane & 3;
  for (int k = 0; k < ks; ++k) {
    const float *xa = X + g * in::kStride + 8 * k + t;
    const float *yb = Y + (8 * k + t) * in::kStride + g;
    const float x[4] = {xa[0], xa[8 * in::kStride], xa[4], xa[8 * in::kStride + 4]};
    const float y[2] = {yb[0], yb[4 * in::kStride]};
    uint32_t xh[4], yh[2];
#pragma unroll
    for (int i = 0; i < 4; ++i) xh[i] = to_tf32(x[i]);
#pragma unroll
    for (int i = 0; i < 2; ++i) yh[i] = to_tf32(y[i]);
    if constexpr (kExact) {
      uint32_t xl[4], yl[2];
#pragma unroll
      for (int i = 0; i < 4; ++i) xl[i] = to_tf32(x[i] - __uint_as_float(xh[i]));
#pragma unroll
      for (int i = 0; i < 2; ++i) yl[i] = to_tf32(y[i] - __uint_as_float(yh[i]));
      mma_1688_tf32(d, xl[0], xl[1], xl[2], xl[3], yh[0], yh[1]);
      mma_1688_tf32(d, xh[0], xh[1], xh[2], xh[3], yl[0], yl[1]);
    }
    mma_1688_tf32(d, xh[0], xh[1], xh[2], xh[3], yh[0], yh[1]);
  }
}
__device__ __forceinline__ void st_tile(float *D, const float (&d)[4], float sgn, int lane) {
  const int g = lane >> 2, t = lane & 3;
  *reinterpret_cast<float2 *>(D + g * in::kStride + 2 * t) = make_float2(sgn * d[0], sgn * d[1]);
  *reinterpret_cast<float2 *>(D + (g + 8) * in::kStride + 2 * t) = make_float2(sgn * d[2], sgn * d[3]);
}
// the same tile, times sgn and the column's beta, into T hi and T lo (rows row0.., columns col0..)
__device__ __forceinline__ void st_tile_t(uint8_t *blk, int row0, int col0, const float (&d)[4], float sgn,
                                          const float *s_beta, int lane) {
  const int g = lane >> 2, c = col0 + 2 * (lane & 3);
  const float b0 = sgn * s_beta[c], b1 = sgn * s_beta[c + 1];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    uint32_t hi, lo;
    split2(d[2 * i] * b0, d[2 * i + 1] * b1, hi, lo);
    const uint32_t off = swz_offset(64, row0 + g + 8 * i, c);
    *reinterpret_cast<uint32_t *>(blk + off) = hi;
    *reinterpret_cast<uint32_t *>(blk + kBlkTlo + off) = lo;
  }
}

// One CTA per (chunk slot, key head): the products of the chunk's keys and queries serve every value head of the group.
// Bound by latency (short dependent phases on one chunk), hidden by three CTAs per SM; its traffic is the keys and
// queries in and 25 KB a value head out.
__global__ void __launch_bounds__(in::kThreads, 3) gdn_intra_kernel(const __grid_constant__ GdnPrefillParams prm) {
  using namespace in;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t *small = sm + OFF_SMALL;
  float *s_norm = reinterpret_cast<float *>(small + SM_NORM);
  float *s_beta = reinterpret_cast<float *>(small + SM_BETA);
  float *s_bi = reinterpret_cast<float *>(small + SM_BI);
  float *s_bf = reinterpret_cast<float *>(small + SM_BF);
  uint64_t *bar_in = reinterpret_cast<uint64_t *>(small + SM_BAR);
  uint64_t *bar_mma = bar_in + 1;
  uint32_t *s_tmem = reinterpret_cast<uint32_t *>(small + SM_TMEM);
  volatile uint32_t *s_abort = reinterpret_cast<volatile uint32_t *>(small + SM_ABORT);
  uint8_t *s_blk = sm + OFF_BLK;
  float *sA = reinterpret_cast<float *>(sm + OFF_A), *sP = reinterpret_cast<float *>(sm + OFF_P);

  grid_launch_dependents();   // the state pass may take SMs as this grid leaves them
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int hk = blockIdx.x % prm.Hk, slot = blockIdx.x / prm.Hk;
  int n = 0;   // the slot's sequence: the last that starts at or before it
  for (int hi = prm.num_seqs - 1; n < hi;) {
    const int mid = (n + hi + 1) >> 1;
    if (first_slot(prm, mid) <= slot) n = mid; else hi = mid - 1;
  }
  const int tok0 = prm.cu[n] + (slot - first_slot(prm, n)) * kC;
  const int valid = min(kC, prm.cu[n + 1] - tok0);
  if (valid <= 0) return;   // a slot between two sequences

  if (tid == 0) {
    mbar_init(bar_in, 1);
    mbar_init(bar_mma, 1);
    *s_abort = 0;
    fence_mbar_init();
    mbar_arrive_expect_tx(bar_in, 32768);
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      tma_load_3d(sm + OFF_KQ + 16384 * x, &prm.tk, 64 * x, hk, tok0, bar_in);
      tma_load_3d(sm + OFF_KQ + 16384 * x + 8192, &prm.tq, 64 * x, hk, tok0, bar_in);
    }
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
  if (tid == 0) {
    wait_or_abort(bar_in, 0, s_abort, prm.status);
    const uint64_t kq = desc_kmajor_base(smem_u32(sm + OFF_KQ));
    const uint32_t id = idesc_bf16(128, 128, false, false);
#pragma unroll
    for (int s = 0; s < 8; ++s) mma_bf16(tmem, kq + kmajor_step(128, s), kq + kmajor_step(128, s), id, s > 0);
    mma_commit(bar_mma);
  }
  __syncwarp();
  const int q4 = warp & 3, ib = warp >> 2;   // TMEM lane quadrant, half of the 64 key columns
  const uint32_t lanes = tmem + (static_cast<uint32_t>(q4 * 32) << 16);

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
        b[e] = lam == lam ? static_cast<int64_t>(rintf(lam)) * 4294967296ll +
                                static_cast<int64_t>((lam - rintf(lam)) * 4294967296.0f)
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
        s_bi[2 * lane + e] = static_cast<float>(static_cast<int>(x >> 32));
        s_bf[2 * lane + e] = static_cast<float>(static_cast<uint32_t>(x)) * 2.3283064365386963e-10f;
      }
    }
    if (gh == 0) {
      wait_or_abort(bar_mma, 0, s_abort, prm.status);
      tc_fence_after();
      if (warp < 4) {   // row 32 q4 + lane: its diagonal entry
        uint32_t v[32];
        tmem_ld16_async(lanes + 32 * q4, v);
        tmem_ld16_async(lanes + 32 * q4 + 16, v + 16);
        tmem_wait_ld();
        tmem_tie<32>(v);
        float d = 0.f;
#pragma unroll
        for (int e = 0; e < 32; ++e) d = e == lane ? __uint_as_float(v[e]) : d;
        const int r = 32 * q4 + lane;
        s_norm[r] = (r & 63) < valid ? rsqrtf(d + kL2Eps) : 0.f;
      }
    }
    __syncthreads();

    // ---- A and P (fp32) from TMEM; the block's factors
    {
      const bool is_p = q4 >= 2;
      const int r = (q4 & 1) * 32 + lane;
      const float bi = s_bi[r], bf = s_bf[r];
      const float rowf = is_p ? prm.scale * s_norm[64 + r] : s_beta[r] * s_norm[r];
      float *dst = (is_p ? sP : sA) + r * kStride + 32 * ib;
      if ((q4 & 1) < ib) {   // rows 0..31, columns 32..63: above the diagonal
#pragma unroll
        for (int e = 0; e < 32; e += 4) *reinterpret_cast<float4 *>(dst + e) = make_float4(0.f, 0.f, 0.f, 0.f);
      } else {
        const int lim = r < valid ? r - 32 * ib + (is_p ? 1 : 0) : 0;   // kept: i < r (A), i <= r (P)
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          uint32_t v[16];
          tmem_ld16_async(lanes + 32 * ib + 16 * half, v);
          tmem_wait_ld();
          tmem_tie<16>(v);
          float x[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const int i = 32 * ib + 16 * half + e;
            const float dec = fast_exp2((bi - s_bi[i]) + (bf - s_bf[i]));
            x[e] = 16 * half + e < lim ? __uint_as_float(v[e]) * (rowf * s_norm[i]) * dec : 0.f;
          }
#pragma unroll
          for (int e = 0; e < 16; e += 4)
            *reinterpret_cast<float4 *>(dst + 16 * half + e) = make_float4(x[e], x[e + 1], x[e + 2], x[e + 3]);
        }
      }
      if (tid < 64) {
        float *vec = reinterpret_cast<float *>(s_blk + kBlkVec);
        const float eb = fast_exp2(s_bi[tid]) * fast_exp2(s_bf[tid]);
        vec[kVecK + tid] = s_norm[tid] * eb;
        vec[kVecQ + tid] = prm.scale * s_norm[64 + tid] * eb;
        vec[kVecS + tid] = s_norm[tid] * fast_exp2((s_bi[63] - s_bi[tid]) + (s_bf[63] - s_bf[tid]));
        if (tid == 63) vec[kVecGamma] = eb;
      }
    }
    // zeros above the diagonal of T hi, T lo, P T: 6 blocks x 16 rows x two 16-byte pieces of each
    for (int x = tid; x < 3 * 192; x += kThreads) {
      const int which = x / 192, y = x % 192, b6 = y >> 5, rr = (y >> 1) & 15, hc = y & 1;
      const int I = b6 < 3 ? 0 : b6 < 5 ? 1 : 2;
      const int J = b6 < 3 ? b6 + 1 : b6 < 5 ? b6 - 1 : 3;
      uint8_t *tile = s_blk + (which == 0 ? 0u : which == 1 ? kBlkTlo : 8192u);
      *reinterpret_cast<uint4 *>(tile + swz_offset(64, 16 * I + rr, 16 * J + 8 * hc)) = make_uint4(0, 0, 0, 0);
    }
    __syncthreads();

    // ---- T = (I + A)^-1 Diag(beta): 16 x 16 diagonal inverses D_R by substitution, then
    //   L^-1_10 = -D_1 A_10 D_0,  L^-1_32 = -D_3 A_32 D_2,  L^-1 (rows 32.., cols ..31) = -I_2 A_(23,01) I_1
    // in place in the A tile, temporaries in its unused upper part; every block goes to T hi / T lo as it is made.
    {
      // task (block R, column jc): lane q = lane % 4 of it carries rows q, q + 4, q + 8, q + 12
      const int q = lane & 3, jc = 8 * (warp & 1) + (lane >> 2), R = warp >> 1;
      const float *a = sA + (16 * R) * kStride + 16 * R;
      float xs[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) xs[i] = 4 * i + q == jc ? 1.f : 0.f;
#pragma unroll
      for (int m = 0; m < 15; ++m) {
        const float xm = __shfl_sync(0xffffffffu, xs[m >> 2], (lane & ~3) | (m & 3));
#pragma unroll
        for (int i = (m + 1) >> 2; i < 4; ++i) {
          const int r = 4 * i + q;
          if (r > m) xs[i] = fmaf(-a[r * kStride + m], xm, xs[i]);
        }
      }
      switch (R) {   // both warps of the block have read its entries of A
        case 0: named_bar_sync<1>(64); break;
        case 1: named_bar_sync<2>(64); break;
        case 2: named_bar_sync<3>(64); break;
        default: named_bar_sync<4>(64); break;
      }
      const float bc = s_beta[16 * R + jc];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = 16 * R + 4 * i + q, c = 16 * R + jc;
        sA[r * kStride + c] = xs[i];
        const float x = xs[i] * bc;
        const uint16_t hi = f32_to_bf16_bits(x);
        *reinterpret_cast<uint16_t *>(s_blk + swz_offset(64, r, c)) = hi;
        *reinterpret_cast<uint16_t *>(s_blk + kBlkTlo + swz_offset(64, r, c)) = f32_to_bf16_bits(x - bf16_bits_to_f32(hi));
      }
    }
    __syncthreads();
    if (warp < 4) {
      const int lo = warp < 2 ? 0 : 32, nj = warp & 1;
      float d[4] = {0.f, 0.f, 0.f, 0.f};
      mm_tile<true>(d, sA + (lo + 16) * kStride + lo, sA + lo * kStride + lo + 8 * nj, 2, lane);
      st_tile(sA + lo * kStride + lo + 16 + 8 * nj, d, 1.f, lane);
      if (warp < 2) named_bar_sync<5>(64); else named_bar_sync<6>(64);   // A_10 (A_32) has been read
      float e[4] = {0.f, 0.f, 0.f, 0.f};
      mm_tile<true>(e, sA + (lo + 16) * kStride + lo + 16, sA + lo * kStride + lo + 16 + 8 * nj, 2, lane);
      st_tile(sA + (lo + 16) * kStride + lo + 8 * nj, e, -1.f, lane);
      st_tile_t(s_blk, lo + 16, lo + 8 * nj, e, -1.f, s_beta, lane);
    }
    __syncthreads();
    {   // Z = A_(23,01) I_1 -> rows 0..31, cols 32..63
      const int mi = warp >> 2, nj = warp & 3, k0 = nj < 2 ? 0 : 16;
      float d[4] = {0.f, 0.f, 0.f, 0.f};
      mm_tile<true>(d, sA + (32 + 16 * mi) * kStride + k0, sA + k0 * kStride + 8 * nj, (32 - k0) / 8, lane);
      st_tile(sA + (16 * mi) * kStride + 32 + 8 * nj, d, 1.f, lane);
    }
    __syncthreads();
    {
      const int mi = warp >> 2, nj = warp & 3;
      float d[4] = {0.f, 0.f, 0.f, 0.f};
      mm_tile<true>(d, sA + (32 + 16 * mi) * kStride + 32, sA + 32 + 8 * nj, mi ? 4 : 2, lane);
      st_tile(sA + (32 + 16 * mi) * kStride + 8 * nj, d, -1.f, lane);
      st_tile_t(s_blk, 32 + 16 * mi, 8 * nj, d, -1.f, s_beta, lane);
    }
    __syncthreads();
    // ---- P T: 20 tiles of 16 x 8 on and below the diagonal, ten 8-deep steps a warp; an entry is rounded once, to
    // bf16, like the output it goes into
    {
      // (row block, column tile) of each task, 3 bits each; 077: none
      static constexpr uint16_t kTasks[8][4] = {{030, 012, 077, 077}, {031, 013, 077, 077}, {032, 022, 077, 077}, {033, 023, 077, 077},
                                                {020, 034, 077, 077}, {021, 035, 077, 077}, {010, 036, 024, 000}, {011, 037, 025, 001}};
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const int task = kTasks[warp][x];
        if (task == 077) break;
        const int I = task >> 3, cb = task & 7, k0 = 16 * (cb >> 1);
        float d[4] = {0.f, 0.f, 0.f, 0.f};
        mm_tile<false>(d, sP + 16 * I * kStride + k0, sA + k0 * kStride + 8 * cb, (16 * (I + 1) - k0) / 8, lane);
        const int g = lane >> 2, c = 8 * cb + 2 * (lane & 3);
        const float b0 = s_beta[c], b1 = s_beta[c + 1];
        *reinterpret_cast<uint32_t *>(s_blk + 8192 + swz_offset(64, 16 * I + g, c)) = pack_bf16x2(d[0] * b0, d[1] * b1);
        *reinterpret_cast<uint32_t *>(s_blk + 8192 + swz_offset(64, 16 * I + g + 8, c)) = pack_bf16x2(d[2] * b0, d[3] * b1);
      }
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
// CTA = (sequence, value head) with kG groups, each owning 64 of the value channels, or (sequence, value head, half)
// with one.  A group is 8 epilogue warps (warp w: TMEM lanes 32 (w % 4).., 32 of the 64 columns) and one issuing warp;
// one more warp feeds both groups' chunks through two stages.  With [. | .] hi and lo side by side, a chunk is
//   D  = [k ; q] [S | S]                       (M = 128: keys' and queries' rows; N = 128; K = 128)
//   R  = v - e^b/|k| (k S)                     (warps of lanes 0..63; q S waits in the others' registers)
//   D  = [T ; P T] [R | R],  X = T_lo R_hi     (N = 128 and 64, K = 64 tokens)
//   U' = e^(b_63 - b)/|k| (T R), o = scale e^b/|q| (q S) + P T R
//   D  = k^T [U' | U'],  S = e^(b_63) S + D    (M = 128 key channels; S in registers, 32 a thread)
// The serial path of a chunk is three products and three short epilogues; two groups on an SM fill each other's gaps.
namespace ch {
template <int kG>
struct Map {
  static constexpr int kThreads = 32 * (8 * kG + kG + 1);
  static constexpr uint32_t ST_BLK = 32768, ST_V = ST_BLK + kGdnBlkBytes, kStage = ST_V + 8192 * kG;
  static constexpr uint32_t OFF_RLO = 2 * kStage, OFF_S = OFF_RLO + 8192 * kG, OFF_SMALL = OFF_S + 32768 * kG;
  static constexpr uint32_t SM_BAR = 0 /* full[2], empty[2], then m1, m2, m3 of each group */, SM_TMEM = 96, SM_ABORT = 100,
                            SM_END = 128;
  static constexpr uint32_t kSmemBytes = OFF_SMALL + SM_END;
  static constexpr uint32_t kTmemCols = 256 * kG;
  static_assert(kSmemBytes <= 232448 && kStage % 1024 == 0 && OFF_S % 1024 == 0, "shared memory map");
};
constexpr uint32_t TM_X = 128;   // columns of a group: D (128), X (64)
}  // namespace ch

__device__ __forceinline__ void bar_arrive(int id, int count) { asm volatile("bar.arrive %0, %1;" ::"r"(id), "r"(count) : "memory"); }
__device__ __forceinline__ void bar_wait(int id, int count) { asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(count) : "memory"); }

template <int kG>
__global__ void __launch_bounds__(ch::Map<kG>::kThreads, 1) gdn_chain_kernel(const __grid_constant__ GdnPrefillParams prm) {
  using M = ch::Map<kG>;
  extern __shared__ __align__(1024) uint8_t sm[];
  uint8_t *small = sm + M::OFF_SMALL;
  uint64_t *bar_full = reinterpret_cast<uint64_t *>(small + M::SM_BAR), *bar_empty = bar_full + 2, *bar_m = bar_full + 4;
  uint32_t *s_tmem = reinterpret_cast<uint32_t *>(small + M::SM_TMEM);
  volatile uint32_t *s_abort = reinterpret_cast<volatile uint32_t *>(small + M::SM_ABORT);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  constexpr int kIssuer0 = 8 * kG, kProducer = 9 * kG;   // warps
  if (smem_u32(sm) & 1023u) {   // operand tiles need the alignment declared above
    if (tid == 0) {
      atomicOr(prm.status, KDA_DEVICE_TIMEOUT);
      grid_dependency_wait();
    }
    return;
  }

  const int item = kG == 2 ? blockIdx.x : blockIdx.x >> 1;
  const int half0 = kG == 2 ? 0 : blockIdx.x & 1;        // first 64-channel half of this CTA
  const int h = item % prm.Hv, n = prm.order[item / prm.Hv], hk = h / prm.group;
  const int t0 = prm.cu[n], len = prm.cu[n + 1] - t0;
  const int nchunks = (len + kC - 1) / kC;
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
  // epilogue thread: TMEM lane 32 quad + lane, columns cl .. cl + 31 of the group's 64
  const int grp = warp >> 3, quad = warp & 3, cl = 32 * ((warp >> 2) & 1);
  const bool worker = warp < kIssuer0;
  const int row = 32 * quad + lane, v0 = 64 * (half0 + grp) + cl;   // state row (key channel), first value channel
  float S[32];
  if (worker) {
#pragma unroll
    for (int e = 0; e < 32; e += 4) {
      const float4 x = src ? *reinterpret_cast<const float4 *>(src + row * kD + v0 + e) : make_float4(0.f, 0.f, 0.f, 0.f);
      S[e] = x.x; S[e + 1] = x.y; S[e + 2] = x.z; S[e + 3] = x.w;
    }
  }
  if (nchunks > 0) {
    if (tid == 0) {
      for (int i = 0; i < 2; ++i) {
        mbar_init(&bar_full[i], 1);
        mbar_init(&bar_empty[i], 8 * kG);
      }
      for (int i = 0; i < 3 * kG; ++i) mbar_init(&bar_m[i], 1);
      *s_abort = 0;
      fence_mbar_init();
    }
    if (warp == kProducer) {
      tmem_alloc(s_tmem, M::kTmemCols);
      tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *s_tmem;

    if (warp == kProducer) {
      // ------------------------------------------------------------ chunk c's keys, queries, values and block -> stage
      if (lane == 0) {
        const uint8_t *blk = prm.blocks + (static_cast<size_t>(first_slot(prm, n)) * prm.Hv + h) * kGdnBlkBytes;
        const size_t step = static_cast<size_t>(prm.Hv) * kGdnBlkBytes;
        int c = 0;
        for (; c < nchunks && !*s_abort; ++c) {
          const int s = c & 1;
          if (c >= 2) wait_or_abort(&bar_empty[s], ((c >> 1) - 1) & 1, s_abort, prm.status);
          if (*s_abort) break;
          uint8_t *st = sm + s * M::kStage;
          mbar_arrive_expect_tx(&bar_full[s], M::kStage);
          const int tok = t0 + c * kC;
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            tma_load_3d(st + 16384 * x, &prm.tk, 64 * x, hk, tok, &bar_full[s]);
            tma_load_3d(st + 16384 * x + 8192, &prm.tq, 64 * x, hk, tok, &bar_full[s]);
          }
#pragma unroll
          for (int g = 0; g < kG; ++g) tma_load_3d(st + M::ST_V + 8192 * g, &prm.tv, 64 * (half0 + g), h, tok, &bar_full[s]);
          if (c == 0) grid_dependency_wait();   // the blocks are the intra-chunk grid's
          bulk_load(st + M::ST_BLK, blk + c * step, kGdnBlkBytes, &bar_full[s]);
        }
        // the copies that were issued last have landed before the CTA ends, whatever the others found
        for (int i = max(0, c - 2); i < c; ++i) mbar_wait(&bar_full[i & 1], (i >> 1) & 1);
      }
      __syncwarp();
    } else if (!worker) {
      // ------------------------------------------------------------ products of one group
      const int g = warp - kIssuer0, bar = 1 + g;
      uint64_t *m = bar_m + 3 * g;
      const uint32_t d = tmem + 256 * g, x = d + ch::TM_X;
      const uint64_t s_desc = desc_mnmajor_base(smem_u32(sm + M::OFF_S + 32768 * g), 128);
      const uint32_t rlo = smem_u32(sm + M::OFF_RLO + 8192 * g);
      for (int c = 0; c < nchunks; ++c) {
        uint8_t *st = sm + (c & 1) * M::kStage;
        const uint32_t rhi = smem_u32(st + M::ST_V + 8192 * g);
        const uint64_t kq = desc_kmajor_base(smem_u32(st)), kt = desc_mnmajor_base(smem_u32(st), 128);
        const uint64_t tp = desc_kmajor_base(smem_u32(st + M::ST_BLK)), tl = desc_kmajor_base(smem_u32(st + M::ST_BLK + kBlkTlo));
        const uint64_t r2 = smem_desc(rhi, rlo - rhi, 1024);
        bar_wait(bar, 288);   // S is in place
        if (lane == 0) {
          wait_or_abort(&bar_full[c & 1], (c >> 1) & 1, s_abort, prm.status);
          tc_fence_after();
          const uint32_t id = idesc_bf16(128, 128, false, true);
#pragma unroll
          for (int k = 0; k < 8; ++k) mma_bf16(d, kq + kmajor_step(128, k), s_desc + mnmajor_step(k), id, k > 0);
          mma_commit(&m[0]);
        }
        __syncwarp();
        bar_wait(bar, 288);   // R is in place, D has been read
        if (lane == 0) {
          tc_fence_after();
          const uint32_t id = idesc_bf16(128, 128, false, true), id1 = idesc_bf16(128, 64, false, true);
#pragma unroll
          for (int k = 0; k < 4; ++k) mma_bf16(d, tp + kmajor_step(128, k), r2 + mnmajor_step(k), id, k > 0);
#pragma unroll
          for (int k = 0; k < 4; ++k) mma_bf16(x, tl + kmajor_step(128, k), r2 + mnmajor_step(k), id1, k > 0);
          mma_commit(&m[1]);
        }
        __syncwarp();
        bar_wait(bar, 288);   // U' is in place, D has been read
        if (lane == 0) {
          tc_fence_after();
          const uint32_t id = idesc_bf16(128, 128, true, true);
#pragma unroll
          for (int k = 0; k < 4; ++k) mma_bf16(d, kt + mnmajor_step(k), r2 + mnmajor_step(k), id, k > 0);
          mma_commit(&m[2]);
        }
        __syncwarp();
      }
    } else {
      // ------------------------------------------------------------ epilogues of one group
      const int bar = 1 + grp;
      uint64_t *m = bar_m + 3 * grp;
      const uint32_t d = tmem + 256 * grp + (static_cast<uint32_t>(quad * 32) << 16) + cl, x = d + ch::TM_X;
      uint8_t *s_tile = sm + M::OFF_S + 32768 * grp, *rlo = sm + M::OFF_RLO + 8192 * grp;
      // 8 fp32 values -> 16 bytes of hi and of lo, columns c.. of row r (tiles of R rows)
      auto put8 = [](uint8_t *hi_tile, uint8_t *lo_tile, uint32_t off, const float *f) {
        uint4 hi, lo;
        split2(f[0], f[1], hi.x, lo.x);
        split2(f[2], f[3], hi.y, lo.y);
        split2(f[4], f[5], hi.z, lo.z);
        split2(f[6], f[7], hi.w, lo.w);
        *reinterpret_cast<uint4 *>(hi_tile + off) = hi;
        *reinterpret_cast<uint4 *>(lo_tile + off) = lo;
      };
      auto store_s = [&] {
#pragma unroll
        for (int e = 0; e < 32; e += 8) put8(s_tile, s_tile + 16384, swz_offset(128, row, cl + e), S + e);
        fence_async_smem();
        tc_fence_before();
        bar_arrive(bar, 288);
      };
      // 16 columns of D, hi and lo part added
      auto load16 = [&](int e, float *f) {
        uint32_t a[16], b[16];
        tmem_ld16_async(d + e, a);
        tmem_ld16_async(d + 64 + e, b);
        tmem_wait_ld();
        tmem_tie<16>(a);
        tmem_tie<16>(b);
#pragma unroll
        for (int i = 0; i < 16; ++i) f[i] = __uint_as_float(a[i]) + __uint_as_float(b[i]);
      };
      store_s();
      for (int c = 0; c < nchunks; ++c) {
        uint8_t *st = sm + (c & 1) * M::kStage;
        uint8_t *rhi = st + M::ST_V + 8192 * grp;
        const float *vec = reinterpret_cast<const float *>(st + M::ST_BLK + kBlkVec);
        const int valid = min(kC, len - c * kC);
        wait_or_abort(&bar_full[c & 1], (c >> 1) & 1, s_abort, prm.status);
        // keys behind the sequence's end may hold anything; their U' is 0, but 0 x NaN is not (each group clears them
        // for its own last product; no other product's result there is used)
        if (valid < kC)
          for (int i = tid & 255; i < (kC - valid) * 16; i += 256)
            *reinterpret_cast<uint4 *>(st + swz_offset(128, valid + (i >> 4), 8 * (i & 15))) = make_uint4(0, 0, 0, 0);
        float qs[32];   // lanes 64..127: q S of token row - 64
        wait_or_abort(&m[0], c & 1, s_abort, prm.status);
        tc_fence_after();
        if (quad < 2) {
          const float f = -vec[kVecK + row];
          const bool there = row < valid;
#pragma unroll
          for (int e = 0; e < 32; e += 16) {
            float ks[16];
            load16(e, ks);
#pragma unroll
            for (int y = 0; y < 16; y += 8) {
              const uint32_t off = swz_offset(64, row, cl + e + y);
              const uint4 w = *reinterpret_cast<const uint4 *>(rhi + off);
              const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
              float r[8];
#pragma unroll
              for (int z = 0; z < 4; ++z) {
                const float2 v2 = unpack_bf16x2(ws[z]);
                r[2 * z] = there ? fmaf(f, ks[y + 2 * z], v2.x) : 0.f;
                r[2 * z + 1] = there ? fmaf(f, ks[y + 2 * z + 1], v2.y) : 0.f;
              }
              put8(rhi, rlo, off, r);
            }
          }
        } else {
          load16(0, qs);
          load16(16, qs + 16);
        }
        fence_async_smem();
        tc_fence_before();
        bar_arrive(bar, 288);

        wait_or_abort(&m[1], c & 1, s_abort, prm.status);
        tc_fence_after();
        if (quad < 2) {
          const float f = vec[kVecS + row];
#pragma unroll
          for (int e = 0; e < 32; e += 16) {
            float u[16];
            uint32_t w[16];
            tmem_ld16_async(x + e, w);
            load16(e, u);
            tmem_tie<16>(w);
#pragma unroll
            for (int i = 0; i < 16; ++i) u[i] = f * (u[i] + __uint_as_float(w[i]));
            put8(rhi, rlo, swz_offset(64, row, cl + e), u);
            put8(rhi, rlo, swz_offset(64, row, cl + e + 8), u + 8);
          }
          fence_async_smem();
          tc_fence_before();
          bar_arrive(bar, 288);
        } else {
          const float f = vec[kVecQ + row - 64];
#pragma unroll
          for (int e = 0; e < 32; e += 16) {
            float u[16];
            load16(e, u);
#pragma unroll
            for (int i = 0; i < 16; ++i) qs[e + i] = fmaf(f, qs[e + i], u[i]);
          }
          tc_fence_before();
          bar_arrive(bar, 288);
          if (row - 64 < valid) {
            uint16_t *o = prm.out + static_cast<int64_t>(t0 + c * kC + row - 64) * prm.out_stride + h * kD + v0;
#pragma unroll
            for (int e = 0; e < 32; e += 8)
              *reinterpret_cast<uint4 *>(o + e) = make_uint4(pack_bf16x2(qs[e], qs[e + 1]), pack_bf16x2(qs[e + 2], qs[e + 3]),
                                                             pack_bf16x2(qs[e + 4], qs[e + 5]), pack_bf16x2(qs[e + 6], qs[e + 7]));
          }
        }

        const float gamma = vec[kVecGamma];
        wait_or_abort(&m[2], c & 1, s_abort, prm.status);
        tc_fence_after();
#pragma unroll
        for (int e = 0; e < 32; e += 16) {
          float u[16];
          load16(e, u);
#pragma unroll
          for (int i = 0; i < 16; ++i) S[e + i] = fmaf(gamma, S[e + i], u[i]);
        }
        if (c + 1 < nchunks) store_s();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar_empty[c & 1]);
      }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kProducer) {
      tc_fence_after();
      tmem_dealloc(tmem, M::kTmemCols);
    }
  }
  if (nchunks == 0 && tid == 0) grid_dependency_wait();
  if (worker) {
#pragma unroll
    for (int e = 0; e < 32; e += 4)
      *reinterpret_cast<float4 *>(dst + row * kD + v0 + e) = make_float4(S[e], S[e + 1], S[e + 2], S[e + 3]);
  }
}

template <int kG>
cudaError_t launch_chain(const GdnPrefillParams &p, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(p.num_seqs) * p.Hv * (kG == 2 ? 1 : 2));
  cfg.blockDim = dim3(ch::Map<kG>::kThreads);
  cfg.dynamicSmemBytes = ch::Map<kG>::kSmemBytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, gdn_chain_kernel<kG>, p);
}

}  // namespace

size_t gdn_prefill_workspace_bytes(int64_t total_tokens, int num_seqs, int Hv) {
  return (total_tokens / kC + num_seqs) * static_cast<size_t>(Hv) * kGdnBlkBytes;
}

cudaError_t launch_gdn_prefill(const GdnRecurrentArgs &a, const int32_t *cu_host, int num_seqs, uint8_t *blocks,
                               cudaStream_t stream) {
  static std::mutex mu;
  static uint64_t done = 0;
  if (const cudaError_t e = set_attributes_once(mu, done, [] {
        cudaError_t r = cudaFuncSetAttribute(gdn_intra_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, in::kSmemBytes);
        if (r == cudaSuccess)
          r = cudaFuncSetAttribute(gdn_chain_kernel<1>, cudaFuncAttributeMaxDynamicSharedMemorySize, ch::Map<1>::kSmemBytes);
        if (r == cudaSuccess)
          r = cudaFuncSetAttribute(gdn_chain_kernel<2>, cudaFuncAttributeMaxDynamicSharedMemorySize, ch::Map<2>::kSmemBytes);
        return r;
      }))
    return e;
  int dev = 0, sms = 0;
  if (const cudaError_t e = cudaGetDevice(&dev)) return e;
  if (const cudaError_t e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) return e;
  GdnPrefillParams p;
  const int total = cu_host[num_seqs], Hk = a.Hv / a.group;
  if (!make_token_map(&p.tq, a.q, Hk, total, a.qk_stride) || !make_token_map(&p.tk, a.k, Hk, total, a.qk_stride) ||
      !make_token_map(&p.tv, a.v, a.Hv, total, a.v_stride))
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
    gdn_intra_kernel<<<static_cast<unsigned>(slots) * Hk, in::kThreads, in::kSmemBytes, stream>>>(p);
    if (const cudaError_t e = cudaGetLastError()) return e;
    // one half of the value channels per CTA while that many CTAs have an SM each
    const cudaError_t e = 2ll * ns * a.Hv <= sms ? launch_chain<1>(p, stream) : launch_chain<2>(p, stream);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace kda
