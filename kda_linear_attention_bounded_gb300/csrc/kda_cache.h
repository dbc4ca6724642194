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
struct PrefixGroup {         // of the plan: a group's place in the line of work
  int64_t unit;              // its first
  int64_t piece;             // rows of pieces before its
  int b0, rows, tiles, len;  // first request, rows of a key head, tiles and tokens that are shared (0: none)
  int table_row, pad[3];     // the request whose table row is read
};
struct PrefixPlan {
  int64_t units;
  int stretches;
  int ticket;                // of the own tokens' stretches
};
struct PrefixArgs {
  PagedArgs a;               // own, rows: for the requests' own tokens
  const int32_t *prefix_lens, *group_starts;
  int groups;
  int2 *own;                 // [B]: a request's first own token, its group (-1: nothing is shared)
  PrefixPlan *plan;
  PrefixGroup *group;        // [groups]
  float *pieces;             // rows of kPagedPartFloats
};
// Bytes that the plan, the rows of own tokens and the pieces take behind the paged attention's workspace; with args and base the
// pointers are set, too.
size_t shared_prefix_bytes(int B, int T, int Hq, int Hk, int groups, uint8_t *base, PrefixArgs *args);
cudaError_t launch_shared_prefix(const PrefixArgs &args, cudaStream_t stream);

}  // namespace kda
