// Rotary positions of a step's tokens, the queries turned in place or into another tensor, the keys turned on their way
// into the pages, the values stored beside them.
//
// Frequency f of a token at position p turns its pair of channels by theta = p w_f.  cos and sin need theta modulo 2 pi, and
// fp32 has no bit of it left where p w passes 2^24.  So the angle is kept in turns as a 64-bit fraction of one:
// w_f / 2 pi modulo 1 (24 bits of w times 88 of 1 / 2 pi, off by 2^-64 for w <= 1) times p, whose product wraps where whole
// turns do.  Its 64 bits go to fp32 as a signed number of half turns in [-1, 1), of which sincospif takes the functions.
//
// Bound by HBM: every row is read and written once (9001 tokens of 32 + 2 x 8 heads: 221 MB), and the 64 functions of a token
// serve all of its heads.  A warp takes a token, or a part of its heads where there are few tokens: eight lanes a row, each two of
// the row's 16-byte pieces: those whose channels make pairs (channels f and f + R / 2 lie R / 16 pieces apart, 2 f and 2 f + 1 side by
// side), so that a lane has both of a pair and the same eight frequencies in either layout.
#include "kda_cache.h"
#include "kda_hybrid.cuh"

namespace kda {
namespace {

constexpr int kWarps = 8;

// 1 / 2 pi = 0.28BE60DB9391054A7F09D5F47D4D3770.. (hexadecimal)
constexpr uint64_t kTurnHi = 0x28BE60DB9391054Aull, kTurnLo = 0x7F09D5F47D4D3770ull;

// w / 2 pi modulo 1, times 2^64; ok: w is a number below 2^24 in size.
__device__ __forceinline__ uint64_t turns_per_step(float w, bool &ok) {
  const uint32_t bits = __float_as_uint(w);
  const int e = (bits >> 23) & 255;
  ok = e < 151;
  const uint64_t m = e ? (bits & 0x7FFFFFu) | 0x800000u : bits & 0x7FFFFFu;   // w = m 2^(max(e, 1) - 150)
  const int shift = 150 - max(e, 1);
  // m / 2 pi: 24 bits of whole turns, 64 of their fraction
  const uint64_t carry = __umul64hi(m, kTurnLo), low = m * kTurnHi;
  const uint64_t fraction = low + carry, whole = __umul64hi(m, kTurnHi) + (fraction < low);
  const uint64_t x = shift <= 0 ? fraction : shift < 64 ? fraction >> shift | whole << (64 - shift) : shift < 128 ? whole >> (shift - 64) : 0;
  return bits >> 31 ? 0 - x : x;
}

// m cos and m sin of a phase in turns, times 2^64
__device__ __forceinline__ float2 unit(uint64_t phase, float m) {
  float s, c;
  sincospif(__ll2float_rn(static_cast<int64_t>(phase)) * 0x1p-63f, &s, &c);
  return make_float2(m * c, m * s);
}

__device__ __forceinline__ uint4 load16(const uint16_t *p) { return *reinterpret_cast<const uint4 *>(p); }
__device__ __forceinline__ void store16(uint16_t *p, uint4 x) { *reinterpret_cast<uint4 *>(p) = x; }

__device__ __forceinline__ uint32_t turn_pair(uint32_t x, float2 cs) {
  const float2 v = unpack_bf16x2(x);
  return pack_bf16x2(v.x * cs.x - v.y * cs.y, v.y * cs.x + v.x * cs.y);
}
// two words of a and b channels each
__device__ __forceinline__ void turn_words(uint32_t &a, uint32_t &b, float2 cs0, float2 cs1) {
  const float2 x = unpack_bf16x2(a), y = unpack_bf16x2(b);
  a = pack_bf16x2(x.x * cs0.x - y.x * cs0.y, x.y * cs1.x - y.y * cs1.y);
  b = pack_bf16x2(y.x * cs0.x + x.x * cs0.y, y.y * cs1.x + x.y * cs1.y);
}

__global__ void __launch_bounds__(32 * kWarps) rotary_to_pages_kernel(RotaryArgs p, int parts) {
  __shared__ float2 s_turn[kWarps][64];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t item = static_cast<int64_t>(blockIdx.x) * kWarps + warp;
  const int i = static_cast<int>(item / parts), part = static_cast<int>(item - static_cast<int64_t>(i) * parts);
  sm100::grid_dependency_wait();
  sm100::grid_launch_dependents();
  if (i >= p.tokens) return;   // (no barrier of the CTA below)
  const int64_t slot = p.slots[i];
  const int half = p.R >> 1;
  int32_t pos[2] = {0, 0};
  float w[2] = {0.f, 0.f};
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int f = lane + 32 * j;
    if (f < half) {
      pos[j] = p.positions[static_cast<int>(p.axes[j] >> (2 * lane) & 3) * p.position_stride + i];
      w[j] = p.inv_freq[f];
    }
  }
  if (slot < 0 || slot >= static_cast<int64_t>(p.num_pages) * p.page) {
    if (slot != -1 && part == 0 && lane == 0) atomicOr(p.status, KDA_DEVICE_BAD_SLOT);
    return;
  }
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    bool ok;
    const uint64_t step = turns_per_step(w[j], ok);
    const float2 cs = unit(static_cast<uint64_t>(static_cast<int64_t>(pos[j])) * step, p.mscale);
    s_turn[warp][lane + 32 * j] = ok ? cs : make_float2(NAN, NAN);
  }
  __syncwarp();
  const int u = lane & 7, turned = p.R >> 4;   // units of two pieces; those that turn
  float2 cs[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) cs[j] = s_turn[warp][8 * u + j];
  const bool apart = !p.interleaved && u < turned;   // the pieces are R / 16 apart
  const int c0 = apart ? 8 * u : 16 * u, c1 = apart ? 8 * (u + turned) : 16 * u + 8;
  int64_t pg;
  int tok;
  if (slot < (int64_t(1) << 32)) {
    pg = static_cast<uint32_t>(slot) / static_cast<uint32_t>(p.page);
    tok = static_cast<int>(static_cast<uint32_t>(slot) - static_cast<uint32_t>(pg) * p.page);
  } else {
    pg = slot / p.page;
    tok = static_cast<int>(slot - pg * p.page);
  }
  uint16_t *const k_to = p.k_pages + pg * p.k_page_stride + tok * p.k_token_stride;
  uint16_t *const v_to = p.v_pages + pg * p.v_page_stride + tok * p.v_token_stride;
  const int rows = p.Hq + 2 * p.Hk;
  // rows of four a turn; the warp's turns
  const int turns = (rows + 3) >> 2;
  const int t0 = turns * part / parts, t1 = turns * (part + 1) / parts;
#pragma unroll 2
  for (int t = t0; t < t1; ++t) {
    const int r = 4 * t + (lane >> 3);
    if (r >= rows) break;
    const uint16_t *from;
    uint16_t *to;
    bool turn = u < turned;
    if (r < p.Hq) {
      from = p.q + i * p.q_stride + r * kD;
      to = p.out + i * p.out_stride + r * kD;
    } else if (r < p.Hq + p.Hk) {
      from = p.k + i * p.k_stride + (r - p.Hq) * kD;
      to = k_to + (r - p.Hq) * p.k_head_stride;
    } else {
      from = p.v + i * p.v_stride + (r - p.Hq - p.Hk) * kD;
      to = v_to + (r - p.Hq - p.Hk) * p.v_head_stride;
      turn = false;
    }
    uint4 a = load16(from + c0), b = load16(from + c1);
    if (turn) {
      if (p.interleaved) {
        a.x = turn_pair(a.x, cs[0]); a.y = turn_pair(a.y, cs[1]); a.z = turn_pair(a.z, cs[2]); a.w = turn_pair(a.w, cs[3]);
        b.x = turn_pair(b.x, cs[4]); b.y = turn_pair(b.y, cs[5]); b.z = turn_pair(b.z, cs[6]); b.w = turn_pair(b.w, cs[7]);
      } else {
        turn_words(a.x, b.x, cs[0], cs[1]);
        turn_words(a.y, b.y, cs[2], cs[3]);
        turn_words(a.z, b.z, cs[4], cs[5]);
        turn_words(a.w, b.w, cs[6], cs[7]);
      }
    }
    store16(to + c0, a);
    store16(to + c1, b);
  }
}

}  // namespace

cudaError_t launch_rotary_to_pages(const RotaryArgs &a, cudaStream_t stream) {
  if (a.tokens <= 0) return cudaSuccess;
  // A token's rows are split until there are 64 warps for each SM or one turn of rows is left for each.  (Measured, 9001 tokens of
  // 48 rows: up to 16, 64, 128 and 256 warps 39.7, 38.7, 41.5 and 51.4 us: at first the last wave counts, then the functions, which
  // every warp of a token computes for itself.)
  const int turns = (a.Hq + 2 * a.Hk + 3) / 4;
  int parts = 1;
  while (parts < turns && static_cast<int64_t>(a.tokens) * parts < 152 * 64) parts *= 2;
  parts = parts < turns ? parts : turns;
  const int64_t items = static_cast<int64_t>(a.tokens) * parts;
  return launch_dependent(rotary_to_pages_kernel, static_cast<unsigned>((items + kWarps - 1) / kWarps), 32 * kWarps, 0, stream, a,
                          parts);
}

}  // namespace kda
