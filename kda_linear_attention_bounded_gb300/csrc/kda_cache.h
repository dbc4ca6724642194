// Internal launch interface of the calls around the paged cache (kda_cache_api.cu): rotary positions with the store into
// the pages, the pages' own operations, attention over shared prefixes.
#pragma once

#include "kda_hybrid.h"

namespace kda {

// ---------------------------------------------------------------- rotary positions
constexpr int kMaxAxes = 4;
struct RotaryArgs {
  const uint16_t *q, *k, *v;
  int64_t q_stride, k_stride, v_stride, out_stride;        // tokens (heads contiguous)
  int tokens, Hq, Hk;
  const int32_t *positions;                                // [axes, tokens]
  int64_t position_stride;
  const int64_t *slots;
  const float *inv_freq;                                   // [R / 2]
  uint64_t axes[2];                                        // two bits a frequency
  int R, interleaved;
  float mscale;
  uint16_t *k_pages, *v_pages, *out;
  int64_t k_page_stride, k_token_stride, k_head_stride;    // elements
  int64_t v_page_stride, v_token_stride, v_head_stride;
  int num_pages, page;
  uint32_t *status;
};
cudaError_t launch_rotary_to_pages(const RotaryArgs &args, cudaStream_t stream);

// ---------------------------------------------------------------- pages
struct TableArgs {
  const int32_t *table;      // [B, width], row stride `stride`
  int64_t stride;
  int width, B, page;
  uint32_t *status;
};
struct ForkArgs {
  TableArgs t;
  int32_t *table, *seq_lens;
  const int32_t *parents, *children, *free_pages;
  int forks, num_free;
  int32_t *copy_src, *copy_dst, *pages_used;
};
cudaError_t launch_fork_requests(const ForkArgs &args, cudaStream_t stream);

struct ReleaseArgs {
  TableArgs t;
  int32_t *seq_lens;
  const int32_t *rows;
  int num_rows;
  int32_t *free_pages, *num_free;
  int num_pages;
};
cudaError_t launch_release_requests(const ReleaseArgs &args, cudaStream_t stream);

struct CompactArgs {
  TableArgs t;
  const int32_t *seq_lens;
  int num_pages, room;
  int32_t *new_table, *copy_src, *copy_dst, *free_pages, *num_free;
  int64_t new_stride;
};
cudaError_t launch_compact_pages(const CompactArgs &args, cudaStream_t stream);

cudaError_t launch_copy_pages(const kda_page_buffer *buffers, int num_buffers, int num_pages, const int32_t *src,
                              const int32_t *dst, int count, uint32_t *status, cudaStream_t stream);

// ---------------------------------------------------------------- attention over shared prefixes
struct PrefixArgs {
  PagedArgs a;
  const int32_t *prefix_lens, *group_starts;
  int groups;
  uint8_t *scratch;          // shared_prefix_bytes() behind what the paged attention itself needs
};
cudaError_t launch_shared_prefix(const PrefixArgs &args, cudaStream_t stream);

}  // namespace kda
