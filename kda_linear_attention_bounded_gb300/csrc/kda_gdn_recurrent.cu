// Token-by-token gated delta rule on CUDA cores: single-token decode, speculative verify, and the recurrence over
// whole sequences.
//
// Per value head h (key head h / (Hv / Hk)), with one log-decay per (token, head):
//   lambda = -exp(A_log) softplus(a + dt_bias),  beta = sigmoid(beta_logit),  k^, q^ l2-normalised
//   u   = beta (v - e^lambda S^T k^)
//   o   = scale (e^lambda S^T q^ + (k^ . q^) u)               [= scale S_t^T q^]
//   S_t = e^lambda S + k^ u^T
// so one cross-thread reduction per token serves the correction and the output.
//
// Bound by HBM: per (request, head) 64 KiB of state in and 64 KiB out per recorded state.  The columns of S (value
// channels) are independent, so a CTA of 128 threads owns 128 / kP of them: thread = (four columns, kR rows), every
// row of the slice one or more full 128-byte lines.  Small slices keep many CTAs resident, so that the loads of one
// run under the stores of another and the last wave is short.  Measured (16 heads): quarters of the channels, eight CTAs
// per SM 24.8 us for 64 x 1 tokens (5.4 TB/s) and 53.2 us for 64 x 4 (6.4 TB/s); halves 25.6 and 54.7, eighths 29 to 31
// and 61 us (their rows are half lines).
#include "kda_hybrid.cuh"

namespace kda {
namespace {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
constexpr int kTile = kWarps;   // tokens prepared per prologue pass (one per warp)

// A warp's row over its norm.  Where the squares pass fp32 they are taken of the row times 2^-80 (and the 1e-6 is nothing).
__device__ __forceinline__ float4 unit_row(float4 x) {
  float sq = warp_sum(x.x * x.x + x.y * x.y + x.z * x.z + x.w * x.w), eps = kL2Eps;
  if (sq == INFINITY) {
    constexpr float f = 8.271806125530277e-25f;
    x = make_float4(f * x.x, f * x.y, f * x.z, f * x.w);
    sq = warp_sum(x.x * x.x + x.y * x.y + x.z * x.z + x.w * x.w);
    eps = 0.f;
  }
  const float n = rsqrtf(sq + eps);
  return make_float4(x.x * n, x.y * n, x.z * n, x.w * n);
}

template <int kP>
__global__ void __launch_bounds__(kThreads, 8) gdn_recurrent_kernel(GdnRecurrentArgs p) {
  constexpr int kCols = kD / kP;              // value channels of the CTA
  constexpr int kQuads = kCols / 4;           // threads along a row
  constexpr int kGroups = kThreads / kQuads;  // row groups; group g owns rows g, g + kGroups, ...
  constexpr int kR = kD / kGroups;            // rows per thread
  static_assert(kQuads <= 32, "a row lies within one warp");
  __shared__ __align__(16) float s_k[kTile][kD], s_q[kTile][kD];
  __shared__ __align__(16) float s_v[kTile][kCols];
  __shared__ float s_alpha[kTile], s_beta[kTile], s_kq[kTile];
  __shared__ __align__(16) float s_red[2][kWarps][2][kCols];   // [token parity][warp][k | q][column]

  sm100::grid_dependency_wait();
  sm100::grid_launch_dependents();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int part = blockIdx.x % kP;
  const int h = (blockIdx.x / kP) % p.Hv;
  const int n = blockIdx.x / (kP * p.Hv);
  const int hk = h / p.group;
  const int64_t t_begin = p.cu_seqlens ? p.cu_seqlens[n] : static_cast<int64_t>(n) * p.T;
  const int64_t t_end = p.cu_seqlens ? p.cu_seqlens[n + 1] : static_cast<int64_t>(n + 1) * p.T;

  int slot = 0;
  if (p.slot_ids) {
    slot = p.slot_ids[n];
    if (slot == KDA_PAD_SLOT_ID && p.skip_padding) return;   // padding row of a bucketed batch
    if (slot < 0 || slot >= p.num_slots) {
      if (tid == 0) atomicOr(p.status, KDA_DEVICE_BAD_SLOT);
      return;
    }
  }
  const int quad = tid % kQuads, group = tid / kQuads;
  const int col = part * kCols + quad * 4;   // first of this thread's value channels
  float4 S[kR];
  if (p.state_in) {
    const float *src = p.state_in + (static_cast<size_t>(slot) * p.Hv + h) * kD * kD + col;
#pragma unroll
    for (int i = 0; i < kR; ++i) S[i] = __ldcs(reinterpret_cast<const float4 *>(src + (group + i * kGroups) * kD));
  } else {
#pragma unroll
    for (int i = 0; i < kR; ++i) S[i] = make_float4(0.f, 0.f, 0.f, 0.f);
  }
  const float rate = expf(p.A_log[h]), bias = p.dt_bias[h];

  for (int64_t tile = t_begin; tile < t_end; tile += kTile) {
    const int nt = static_cast<int>(min(static_cast<int64_t>(kTile), t_end - tile));
    if (warp < nt) {   // warp w prepares token tile + w
      const int64_t t = tile + warp;
      const uint2 qr = *reinterpret_cast<const uint2 *>(p.q + t * p.qk_stride + hk * kD + lane * 4);
      const uint2 kr = *reinterpret_cast<const uint2 *>(p.k + t * p.qk_stride + hk * kD + lane * 4);
      const float2 q01 = unpack_bf16x2(qr.x), q23 = unpack_bf16x2(qr.y);
      const float2 k01 = unpack_bf16x2(kr.x), k23 = unpack_bf16x2(kr.y);
      const uint16_t *vp = p.v + t * p.v_stride + h * kD + part * kCols;
      for (int c = lane; c < kCols; c += 32) s_v[warp][c] = bf16_bits_to_f32(vp[c]);
      const float4 qh = unit_row(make_float4(q01.x, q01.y, q23.x, q23.y)), kh = unit_row(make_float4(k01.x, k01.y, k23.x, k23.y));
      const float kq = warp_sum(qh.x * kh.x + qh.y * kh.y + qh.z * kh.z + qh.w * kh.w);
      *reinterpret_cast<float4 *>(&s_q[warp][lane * 4]) = qh;
      *reinterpret_cast<float4 *>(&s_k[warp][lane * 4]) = kh;
      if (lane == 0) {
        s_kq[warp] = kq;
        s_alpha[warp] = expf(-rate * softplus(bf16_bits_to_f32(p.a[t * p.a_stride + h]) + bias));
        s_beta[warp] = 1.0f / (1.0f + expf(-bf16_bits_to_f32(p.beta[t * p.beta_stride + h])));
      }
    }
    __syncthreads();

    for (int s = 0; s < nt; ++s) {
      const int64_t t = tile + s;
      float4 pk = make_float4(0.f, 0.f, 0.f, 0.f), pq = pk;
#pragma unroll
      for (int i = 0; i < kR; ++i) {
        const float kc = s_k[s][group + i * kGroups], qc = s_q[s][group + i * kGroups];
        pk.x = fmaf(S[i].x, kc, pk.x); pk.y = fmaf(S[i].y, kc, pk.y);
        pk.z = fmaf(S[i].z, kc, pk.z); pk.w = fmaf(S[i].w, kc, pk.w);
        pq.x = fmaf(S[i].x, qc, pq.x); pq.y = fmaf(S[i].y, qc, pq.y);
        pq.z = fmaf(S[i].z, qc, pq.z); pq.w = fmaf(S[i].w, qc, pq.w);
      }
#pragma unroll
      for (int o = kQuads; o < 32; o <<= 1) {   // the warp's row groups
        pk.x += __shfl_xor_sync(0xffffffffu, pk.x, o); pk.y += __shfl_xor_sync(0xffffffffu, pk.y, o);
        pk.z += __shfl_xor_sync(0xffffffffu, pk.z, o); pk.w += __shfl_xor_sync(0xffffffffu, pk.w, o);
        pq.x += __shfl_xor_sync(0xffffffffu, pq.x, o); pq.y += __shfl_xor_sync(0xffffffffu, pq.y, o);
        pq.z += __shfl_xor_sync(0xffffffffu, pq.z, o); pq.w += __shfl_xor_sync(0xffffffffu, pq.w, o);
      }
      float (*red)[2][kCols] = s_red[s & 1];   // alternating: the next token's sums never meet this one's readers
      if (lane < kQuads) {
        *reinterpret_cast<float4 *>(&red[warp][0][quad * 4]) = pk;
        *reinterpret_cast<float4 *>(&red[warp][1][quad * 4]) = pq;
      }
      __syncthreads();
      float4 wk = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float4 x = *reinterpret_cast<const float4 *>(&red[w][0][quad * 4]);
        wk.x += x.x; wk.y += x.y; wk.z += x.z; wk.w += x.w;
      }
      const float al = s_alpha[s], be = s_beta[s];
      const float4 vv = *reinterpret_cast<const float4 *>(&s_v[s][quad * 4]);
      const float4 u = make_float4(be * (vv.x - al * wk.x), be * (vv.y - al * wk.y), be * (vv.z - al * wk.z),
                                   be * (vv.w - al * wk.w));
      if (group == 0) {
        float4 wq = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          const float4 x = *reinterpret_cast<const float4 *>(&red[w][1][quad * 4]);
          wq.x += x.x; wq.y += x.y; wq.z += x.z; wq.w += x.w;
        }
        const float kq = s_kq[s];
        *reinterpret_cast<uint2 *>(p.out + t * p.out_stride + h * kD + col) =
            make_uint2(pack_bf16x2(p.scale * (al * wq.x + kq * u.x), p.scale * (al * wq.y + kq * u.y)),
                       pack_bf16x2(p.scale * (al * wq.z + kq * u.z), p.scale * (al * wq.w + kq * u.w)));
      }
      float *rec = p.inter ? p.inter + ((static_cast<size_t>(n) * p.T + (t - t_begin)) * p.Hv + h) * kD * kD + col : nullptr;
#pragma unroll
      for (int i = 0; i < kR; ++i) {
        const float kc = s_k[s][group + i * kGroups];
        S[i].x = fmaf(al, S[i].x, kc * u.x); S[i].y = fmaf(al, S[i].y, kc * u.y);
        S[i].z = fmaf(al, S[i].z, kc * u.z); S[i].w = fmaf(al, S[i].w, kc * u.w);
        if (rec) __stcs(reinterpret_cast<float4 *>(rec + (group + i * kGroups) * kD), S[i]);
      }
    }
    __syncthreads();   // the tile's operands are free
  }

  float *dst = p.state_out_pool    ? p.state_out_pool + (static_cast<size_t>(slot) * p.Hv + h) * kD * kD + col
               : p.state_out_dense ? p.state_out_dense + (static_cast<size_t>(n) * p.Hv + h) * kD * kD + col
                                   : nullptr;
  if (dst) {
#pragma unroll
    for (int i = 0; i < kR; ++i) __stcs(reinterpret_cast<float4 *>(dst + (group + i * kGroups) * kD), S[i]);
  }
}

}  // namespace

cudaError_t launch_gdn_recurrent(const GdnRecurrentArgs &args, int num_items, cudaStream_t stream) {
  if (num_items <= 0) return cudaSuccess;
  const int64_t grid = static_cast<int64_t>(num_items) * args.Hv * 4;
  if (grid > 0x7fffffff) return cudaErrorInvalidValue;
  return launch_dependent(gdn_recurrent_kernel<4>, static_cast<unsigned>(grid), kThreads, 0, stream, args);
}

}  // namespace kda
